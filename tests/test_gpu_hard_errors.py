"""A launch that fails is reported, not sent a second time: the first attempt may have changed the cache."""
import ctypes

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
HIP_ERROR, OPTION_ERROR = 8, 7


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sparse_selection_primitive_amd as lib
    lib.load_library()
    return lib


@pytest.mark.parametrize("status", [HIP_ERROR, OPTION_ERROR])
def test_failed_launch_through_the_native_front(L, monkeypatch, status):
    from sparse_selection_primitive_amd import hard
    L.dispatch_plan(torch.zeros(1, 1, dtype=torch.int32, device="cuda"), 1)  # binds
    if hard._native is None:
        pytest.skip("the native front is not built")
    lib = L.load_library()
    sent, again = [], []
    # a C call that launches nothing and reports the status (its arguments are not looked at)
    fails = ctypes.CFUNCTYPE(ctypes.c_int)(lambda: sent.append(1) or status)
    address = ctypes.cast(fails, ctypes.c_void_p).value
    monkeypatch.setattr(hard, "_call", lambda *a: again.append(1))
    real = [ctypes.cast(getattr(lib, "lapsum_" + name), ctypes.c_void_p).value for name in hard._NATIVE_CALLS]
    k = torch.zeros(1, 2, 20, 64, device="cuda", dtype=torch.bfloat16)
    a = torch.zeros(1, 2, 20, device="cuda")
    n = torch.tensor([20], dtype=torch.int32, device="cuda")
    x = torch.randn(4, 16, device="cuda")
    c = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    offsets, slot, _ = torch.zeros(5, dtype=torch.int32, device="cuda"), c.clone(), None
    w = torch.ones(4, 2, device="cuda")
    rows = torch.randn(8, 16, device="cuda")
    calls = {"cache_evict": lambda: L.cache_evict(k, k.clone(), a, a.int(), n, 5),
             "cache_attend": lambda: L.cache_attend(k.transpose(1, 2)[:, :1].contiguous(), k, k, n, a),
             "route_forward": lambda: L.route_forward(x, 2), "route_backward": lambda: L.route_backward(w, x, c),
             "dispatch_plan": lambda: L.dispatch_plan(c, 4), "dispatch_forward": lambda: L.dispatch_forward(x, slot, offsets),
             "dispatch_backward": lambda: L.dispatch_backward(rows, slot),
             "combine_forward": lambda: L.combine_forward(rows, slot, w),
             "combine_backward": lambda: L.combine_backward(x, rows, slot, w, offsets)}
    try:
        for name, call in calls.items():
            to = list(real)
            to[hard._NATIVE_CALLS.index(name)] = address
            hard._native.bind(*to)
            del sent[:], again[:]
            if status == HIP_ERROR:
                with pytest.raises(L.LapsumError, match=name):
                    call()
                assert len(sent) == 1 and not again, name
            else:  # an argument that is refused: nothing was launched, and hard.py says what is wrong with it
                call()
                assert len(sent) == 1 and len(again) == 1, name
    finally:
        hard._native.bind(*real)

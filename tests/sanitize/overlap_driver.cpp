// Checks which arrays the beam selection and the cache reordering take for overlapping against sets of bytes, over random small
// layouts.  Built and run by tests/test_search_overlaps.py with the host runtime alone: launches are counted here and
// reach no GPU, and addresses are numbers that nothing follows.
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <utility>
#include <vector>

#include "../../sparse_selection_primitive_amd/csrc/hard_internal.hpp"

static int launched = 0;
extern "C" hipError_t hipGetLastError(void) { return hipSuccess; }
namespace lapsum {
hipError_t launch_route_forward(const RouteArgs &, int, hipStream_t) { return hipSuccess; }
hipError_t launch_route_backward(const RouteArgs &, int, hipStream_t) { return hipSuccess; }
int64_t plan_tiles(int64_t) { return 1; }
hipError_t launch_dispatch_plan(const int32_t *, int64_t, int, int32_t *, int32_t *, int32_t *, uint32_t *, hipStream_t) {
  return hipSuccess;
}
hipError_t launch_dispatch_rows(const RowsArgs &, int, hipStream_t) { return hipSuccess; }
hipError_t launch_sum_rows(const RowsArgs &, int, hipStream_t) { return hipSuccess; }
hipError_t launch_combine_backward(const RowsArgs &, int, hipStream_t) { return hipSuccess; }
AttendPlan attend_plan(int64_t, int64_t, int64_t, int64_t, bool, int, bool) { return {}; }
hipError_t launch_attend(const AttendArgs &, int, hipStream_t) { return hipSuccess; }
size_t evict_workspace(int64_t, int64_t, int64_t, int64_t) { return 0; }
hipError_t launch_evict(const EvictArgs &, hipStream_t) { return hipSuccess; }
hipError_t launch_product_rows(const ProductArgs &, int, hipStream_t) { return hipSuccess; }
hipError_t launch_product_weights(const ProductArgs &, int, hipStream_t) { return hipSuccess; }
void beam_parts(int64_t, int64_t, int &chunk, int &chunks) { chunk = 512, chunks = 1; }
hipError_t launch_beam_select(const BeamArgs &, int, hipStream_t) { return ++launched, hipSuccess; }
hipError_t launch_reorder(const ReorderArgs &, hipStream_t) { return ++launched, hipSuccess; }
}  // namespace lapsum

static std::mt19937 rng(1);
static int64_t any(int64_t lo, int64_t hi) { return std::uniform_int_distribution<int64_t>(lo, hi)(rng); }
static const uint64_t kBase = 1 << 20;

using Bytes = std::vector<char>;
static Bytes stretch(uint64_t at, int64_t n) {
  Bytes b(1 << 16, 0);
  std::fill_n(b.begin() + (at - kBase), n, 1);
  return b;
}
static bool meet(const Bytes &a, const Bytes &b) {
  for (size_t i = 0; i < a.size(); ++i)
    if (a[i] && b[i]) return true;
  return false;
}
template <class T>
static T *at(uint64_t a) {
  return reinterpret_cast<T *>(a);
}

struct Side {
  int64_t batch, head, entry;
};
static Side strides(const int64_t (&size)[3], int64_t width) {
  int order[3] = {0, 1, 2};
  std::shuffle(order, order + 3, rng);
  int64_t s[3], span = width;
  for (int d : order) {
    s[d] = size[d] == 1 ? width + 8 * any(0, 9) : span + 8 * (any(0, 2) == 0 ? any(0, 4) : any(0, 1) * width / 8);
    if (size[d] > 1) span += s[d] * (size[d] - 1);
  }
  return {s[0], s[1], s[2]};
}

static int check(bool ok, const char *what, int turn) {
  if (!ok) fprintf(stderr, "FAIL %s, turn %d\n", what, turn);
  return ok ? 0 : 1;
}

static int reorder(int turn, int &refused, int &accepted, int &open) {
  const int64_t size[3] = {any(1, 4), any(1, 3), any(1, 4)}, width = 8 * any(1, 2);
  const Side ks = strides(size, width);
  Side vs = any(0, 3) ? ks : strides(size, width);
  for (int64_t *x : {&vs.batch, &vs.head, &vs.entry}) {
    const int d = (int)(x - &vs.batch);
    if (size[d] == 1 && any(0, 1)) *x = width + 8 * any(0, 9);
  }
  const uint64_t k = kBase + 16 * any(0, 200), v = any(0, 4) ? kBase + 16 * any(0, 200) : k;
  const auto side = [&](uint64_t p, const Side &s) {
    Bytes b(1 << 16, 0);
    for (int64_t i = 0; i < size[0]; ++i)
      for (int64_t j = 0; j < size[1]; ++j)
        for (int64_t l = 0; l < size[2]; ++l)
          std::fill_n(b.begin() + (p - kBase) + 2 * (i * s.batch + j * s.head + l * s.entry), 2 * width, 1);
    return b;
  };
  // mostly far away, so that one pair alone decides
  const auto place = [&](int i) { return any(0, 7) ? kBase + 40000 + 1000 * i : kBase + 4 * any(0, 2000); };
  const int64_t caches = size[0] * 4, entries = size[0] * size[1] * size[2] * 4;
  const uint64_t lengths = place(0), parents = place(1), after = place(2), account = any(0, 2) ? place(3) : 0,
                 positions = any(0, 2) ? place(4) : 0;
  const Bytes kb = side(k, ks), vb = side(v, vs), lb = stretch(lengths, caches), pb = stretch(parents, caches);
  const bool alike = (size[0] == 1 || ks.batch == vs.batch) && (size[1] == 1 || ks.head == vs.head) &&
                     (size[2] == 1 || ks.entry == vs.entry);
  const auto gaps = [&](const Bytes &b) {
    const auto last = std::find(b.rbegin(), b.rend(), 1).base();
    return std::count(std::find(b.begin(), b.end(), 1), last, 0) > 0;
  };
  bool bad = false, shared = meet(kb, vb), known = true;
  if (k == v && alike)
    shared = false;
  else if (!alike && k != v && gaps(kb) && gaps(vb))
    known = false;
  std::vector<Bytes> written = {stretch(after, caches)};
  if (account) written.push_back(stretch(account, entries));
  if (positions) written.push_back(stretch(positions, entries));
  for (size_t i = 0; i < written.size(); ++i) {
    for (size_t j = i + 1; j < written.size(); ++j) bad |= meet(written[i], written[j]);
    for (const Bytes *b : {&kb, &vb, &lb, &pb}) bad |= meet(written[i], *b);
  }
  for (const Bytes *b : {&lb, &pb}) bad |= meet(kb, *b) || meet(vb, *b);
  const lapsum_cache c = {at<void>(k), at<void>(v), LAPSUM_BF16, (int32_t)width, size[0],  size[1],  size[2],
                          ks.batch,    ks.head,     ks.entry,    vs.batch,       vs.head, vs.entry};
  launched = 0;
  const lapsum_status st = lapsum_cache_reorder(&c, any(0, 1) ? size[0] : 1, at<int32_t>(parents), at<int32_t>(lengths),
                                                at<float>(account), at<int32_t>(positions), at<int32_t>(after), nullptr);
  (st == LAPSUM_OK ? accepted : refused) += 1;
  if (!bad && shared && !known) {
    ++open;
    return check(st == LAPSUM_OK || st == LAPSUM_ERR_LAYOUT, "status", turn);
  }
  return check(st == (bad || shared ? LAPSUM_ERR_LAYOUT : LAPSUM_OK) && launched == (st == LAPSUM_OK), "reorder", turn);
}

static int select(int turn, int &refused, int &accepted) {
  const int64_t batch = any(1, 3), beams = any(1, 3), vocab = any(1, 20), stride = vocab + any(0, 30), k = any(1, 5);
  const int32_t dtype = any(0, 1) ? LAPSUM_F32 : LAPSUM_BF16;
  const int64_t type = dtype == LAPSUM_F32 ? 4 : 2, rows = batch * beams, places = batch * k * 4;
  const size_t need = lapsum_beam_select_workspace_bytes(batch, beams, vocab, (int32_t)k);
  const auto place = [&](int i) { return any(0, 3) ? kBase + 40000 + 1000 * i : kBase + 4 * any(0, 500); };
  const uint64_t x = kBase + 4 * any(0, 50), scores = place(0), ended = any(0, 1) ? place(1) : 0, out = place(2),
                 parents = place(3), tokens = place(4), work = any(0, 2) ? kBase + 51200 : kBase + 256 * any(0, 8);
  Bytes xb(1 << 16, 0);
  for (int64_t i = 0; i < rows; ++i) std::fill_n(xb.begin() + (x - kBase) + i * stride * type, vocab * type, 1);
  const Bytes xs = xb, sb = stretch(scores, rows * 4), eb = ended ? stretch(ended, rows) : Bytes(1 << 16, 0);
  const Bytes written[] = {stretch(out, places), stretch(parents, places), stretch(tokens, places),
                           stretch(work, (int64_t)need)};
  bool bad = false;
  for (int i = 0; i < 4; ++i) {
    for (int j = i + 1; j < 4; ++j) bad |= meet(written[i], written[j]);
    for (const Bytes *b : {&xs, &sb, &eb}) bad |= meet(written[i], *b);
  }
  launched = 0;
  const lapsum_status st =
      lapsum_beam_select(at<void>(x), dtype, batch, beams, vocab, stride, at<float>(scores), at<uint8_t>(ended), 0, (int32_t)k,
                         at<float>(out), at<int32_t>(parents), at<int32_t>(tokens), at<void>(work), need, nullptr);
  (st == LAPSUM_OK ? accepted : refused) += 1;
  return check(st == (bad ? LAPSUM_ERR_LAYOUT : LAPSUM_OK) && launched == (st == LAPSUM_OK), "select", turn);
}

int main() {
  int failures = 0, count[4] = {}, open = 0;
  for (int turn = 0; turn < 2000 && failures < 20; ++turn) {
    failures += reorder(turn, count[0], count[1], open);
    failures += select(turn, count[2], count[3]);
  }
  printf("reorder: %d refused, %d accepted, %d left to the caller; select: %d refused, %d accepted\n", count[0], count[1], open,
         count[2], count[3]);
  for (int c : count) failures += c < 200;
  failures += open > 200;
  if (failures) return 1;
  printf("all checks passed\n");
  return 0;
}

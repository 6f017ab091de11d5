/* Drives the host side of the experts' products, the beam selection and the cache reordering (argument checks,
 * workspace sizes, early error returns) over a grid of shapes and layouts.  Built and run by
 * tests/test_search_sanitize.py against a host-only AddressSanitizer +
 * UndefinedBehaviorSanitizer build of the library; no call here reaches the GPU: every one lacks an output.  Exits
 * non-zero on the first unexpected status. */
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "lapsum.h"

static int failures = 0;

#define EXPECT(cond, ...)                                        \
    do {                                                         \
        if (!(cond)) {                                           \
            fprintf(stderr, "FAIL %s:%d: ", __FILE__, __LINE__); \
            fprintf(stderr, __VA_ARGS__);                        \
            fprintf(stderr, "\n");                               \
            ++failures;                                          \
        }                                                        \
    } while (0)

static char at[4096] __attribute__((aligned(256)));

static void products(void) {
    const int64_t sizes[] = {-1, 0, 1, 7, 64, 1032, (int64_t)1 << 20, ((int64_t)1 << 20) + 1, INT64_MAX};
    const int64_t rows_list[] = {INT64_MIN, 0, 1, 1000, LAPSUM_MAX_PAIRS, LAPSUM_MAX_PAIRS + 1, INT64_MAX};
    for (size_t i = 0; i < sizeof sizes / sizeof *sizes; ++i)
        for (size_t j = 0; j < sizeof sizes / sizeof *sizes; ++j)
            for (size_t r = 0; r < sizeof rows_list / sizeof *rows_list; ++r)
                for (int turned = 0; turned < 2; ++turned) {
                    const int64_t n = sizes[i], m = sizes[j], rows = rows_list[r];
                    lapsum_experts w = {at, LAPSUM_BF16, 0, 8, n, m, 0, turned ? 1 : m, turned ? n : 1};
                    const int fine = n >= 1 && n <= LAPSUM_MAX_EXPERT_WIDTH && m >= 1 && m <= LAPSUM_MAX_EXPERT_WIDTH &&
                                     rows >= 1 && rows <= LAPSUM_MAX_PAIRS;
                    const int32_t *o = (const int32_t *)at;
                    lapsum_status st = lapsum_expert_product_forward(at, n, rows, &w, o, NULL, NULL);
                    EXPECT(fine ? st == LAPSUM_ERR_NULL : st == LAPSUM_ERR_SHAPE, "forward %lld %lld %lld: %d",
                           (long long)n, (long long)m, (long long)rows, (int)st);
                    st = lapsum_expert_product_backward_rows(at, m, rows, &w, o, NULL, NULL);
                    EXPECT(fine ? st == LAPSUM_ERR_NULL : st == LAPSUM_ERR_SHAPE, "rows: %d", (int)st);
                    st = lapsum_expert_product_backward_weights(at, n, at, m, rows, NULL, &w, NULL);
                    EXPECT(fine ? st == LAPSUM_ERR_NULL : st == LAPSUM_ERR_SHAPE, "weights: %d", (int)st);
                    st = lapsum_expert_product_backward_weights(at, n, at, m, rows, o, &w, NULL);
                    if (fine) EXPECT(st == LAPSUM_ERR_LAYOUT, "matrices in one place: %d", (int)st);
                }
    const int64_t strides[] = {INT64_MIN, -8, 0, 63, LAPSUM_MAX_EXPERT_STRIDE + 1, INT64_MAX};
    for (size_t i = 0; i < sizeof strides / sizeof *strides; ++i) {
        lapsum_experts w = {at, LAPSUM_F16, 0, 8, 64, 64, 4096, strides[i], 1};
        EXPECT(lapsum_expert_product_forward(at, 64, 4, &w, (const int32_t *)at, at, NULL) == LAPSUM_ERR_LAYOUT,
               "matrix stride %lld", (long long)strides[i]);
        w.stride_input = 64;
        EXPECT(lapsum_expert_product_forward(at, strides[i], 4, &w, (const int32_t *)at, at, NULL) ==
                   LAPSUM_ERR_LAYOUT, "row stride %lld", (long long)strides[i]);
    }
    EXPECT(lapsum_expert_product_backward_rows(at, 64, 4, NULL, (const int32_t *)at, at, NULL) == LAPSUM_ERR_NULL, "none");
}

static void beams(void) {
    const int64_t batches[] = {INT64_MIN, 0, 1, 70000, (int64_t)1 << 24, INT64_MAX};
    const int64_t beams_list[] = {-1, 0, 1, 5, 64, 65, INT64_MAX};
    const int64_t vocabs[] = {-1, 0, 1, 511, 512, 50021, LAPSUM_MAX_VOCAB, LAPSUM_MAX_VOCAB + 1, INT64_MAX};
    for (size_t b = 0; b < sizeof batches / sizeof *batches; ++b)
        for (size_t n = 0; n < sizeof beams_list / sizeof *beams_list; ++n)
            for (size_t v = 0; v < sizeof vocabs / sizeof *vocabs; ++v)
                for (int k = -1; k <= 65; k += 11) {
                    const int64_t batch = batches[b], beam = beams_list[n], vocab = vocabs[v];
                    const size_t bytes = lapsum_beam_select_workspace_bytes(batch, beam, vocab, k);
                    const int fine = beam >= 1 && beam <= LAPSUM_MAX_BEAMS && batch >= 1 &&
                                     batch <= LAPSUM_MAX_ROWS / beam && vocab >= 1 && vocab <= LAPSUM_MAX_VOCAB;
                    EXPECT((bytes > 0) == (fine && k >= 1 && k <= LAPSUM_MAX_BEAMS), "bytes %zu", bytes);
                    const lapsum_status st =
                        lapsum_beam_select(at, LAPSUM_BF16, batch, beam, vocab, vocab, (const float *)at, NULL, 0, k,
                                           (float *)(at + 1024), (int32_t *)at, (int32_t *)at, NULL, 0, NULL);
                    EXPECT(st == (!fine ? LAPSUM_ERR_SHAPE : (k < 1 || k > LAPSUM_MAX_BEAMS ? LAPSUM_ERR_OPTION
                                                                                             : LAPSUM_ERR_NULL)),
                           "select %lld %lld %lld %d: %d", (long long)batch, (long long)beam, (long long)vocab, k, (int)st);
                }
}

static void reorder(void) {
    const int64_t beams_list[] = {INT64_MIN, -1, 0, 1, 3, 4, 64, 65, INT64_MAX};
    const int64_t capacities[] = {-1, 0, 1, 100, LAPSUM_MAX_CACHE, LAPSUM_MAX_CACHE + 1, INT64_MAX};
    for (size_t n = 0; n < sizeof beams_list / sizeof *beams_list; ++n)
        for (size_t c = 0; c < sizeof capacities / sizeof *capacities; ++c) {
            const int64_t cap = capacities[c], beam = beams_list[n], head = cap > 0 && cap <= LAPSUM_MAX_CACHE ? cap * 64 : 64;
            lapsum_cache cache = {at, at, LAPSUM_F16, 64, 12, 2, cap, head * 2, head, 64, head * 2, head, 64};
            const lapsum_status st = lapsum_cache_reorder(&cache, beam, (const int32_t *)at, (const int32_t *)at, NULL, NULL,
                                                          NULL, NULL);
            const int fine = cap >= 1 && cap <= LAPSUM_MAX_CACHE && beam >= 1 && beam <= LAPSUM_MAX_BEAMS && 12 % beam == 0;
            EXPECT(st == (fine ? LAPSUM_ERR_NULL : LAPSUM_ERR_SHAPE), "reorder %lld %lld: %d", (long long)beam,
                   (long long)cap, (int)st);
        }
}

int main(void) {
    products();
    beams();
    reorder();
    if (failures) return 1;
    printf("all checks passed\n");
    return 0;
}

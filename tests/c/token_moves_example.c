/* Minimal C99 user of the token moves: sort the choices of a router, send
 * rows to their experts and back (both choices weighted by a half give the
 * rows again), and append one token for each of three sequences to a paged
 * cache.  Exit 0 = ok, 77 = no CUDA device, 1 =
 * failure. */
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include <cuda_runtime.h>

#include "bmmc.h"

#define CHECK(call)                                                                     \
    do {                                                                                \
        const bmmc_status s_ = (call);                                                  \
        if (s_ != BMMC_OK) {                                                            \
            fprintf(stderr, "%s: %s\n", #call, bmmc_status_string(s_));                 \
            return 1;                                                                   \
        }                                                                               \
    } while (0)

/* Memory that host and device both reach. */
static void *both(size_t bytes)
{
    void *p = NULL;
    if (cudaMallocManaged(&p, bytes, cudaMemAttachGlobal) != cudaSuccess) {
        fprintf(stderr, "allocation failed\n");
        exit(1);
    }
    return p;
}

static int experts(void)
{
    enum { T = 5000, K = 2, E = 7, H = 36, N = T * K };
    int32_t *ids = both(N * sizeof *ids), *slot = both(N * sizeof *slot), *source = both(N * sizeof *source);
    int32_t *offsets = both((E + 1) * sizeof *offsets);
    float *x = both(T * H * sizeof *x), *rows = both((size_t)N * H * sizeof *rows), *y = both(T * H * sizeof *y);
    float *w = both(N * sizeof *w);
    size_t need = 0;
    CHECK(expert_sort_workspace(T, K, E, &need));
    void *work = need ? both(need) : NULL;
    for (int i = 0; i < N; ++i) ids[i] = (int32_t)(((uint32_t)i * 2654435761u >> 16) % E), w[i] = 0.5f;
    for (int i = 0; i < T * H; ++i) x[i] = (float)i;
    CHECK(expert_sort(ids, 4, T, K, E, slot, source, offsets, work, need, NULL));
    CHECK(expert_dispatch(x, H, slot, T, K, H, BMMC_F32, rows, H, N, NULL));
    CHECK(expert_combine(rows, H, N, slot, w, BMMC_F32, T, K, H, BMMC_F32, y, H, NULL));
    if (cudaDeviceSynchronize() != cudaSuccess) return 1;
    for (int e = 0; e < E; ++e)
        for (int r = offsets[e]; r < offsets[e + 1]; ++r)
            if (ids[source[r]] != e || slot[source[r]] != r || (r > offsets[e] && source[r] <= source[r - 1])) {
                fprintf(stderr, "row %d is not a row of expert %d\n", r, e);
                return 1;
            }
    if (offsets[0] != 0 || offsets[E] != N) return 1;
    for (int i = 0; i < T * H; ++i)
        if (y[i] != x[i]) {
            fprintf(stderr, "element %d: %f is not %f\n", i, y[i], x[i]);
            return 1;
        }
    return 0;
}

static int append(void)
{
    enum { B = 3, H = 2, D = 4, PAGE = 4, PAGES = 6 };
    float *k = both(B * H * D * sizeof *k), *v = both(B * H * D * sizeof *v);
    float *kc = both(PAGES * PAGE * H * D * sizeof *kc), *vc = both(PAGES * PAGE * H * D * sizeof *vc);
    int32_t *lengths = both(B * sizeof *lengths), *table = both(2 * B * sizeof *table);
    float *freq = both(2 * sizeof *freq);
    const int32_t lens[B] = {0, 3, 5}, pages[2 * B] = {4, -1, 2, -1, 1, 0};
    for (int i = 0; i < B * H * D; ++i) k[i] = v[i] = (float)(i + 1);
    for (int i = 0; i < PAGES * PAGE * H * D; ++i) kc[i] = vc[i] = 0.0f;
    for (int i = 0; i < B; ++i) lengths[i] = lens[i];
    for (int i = 0; i < 2 * B; ++i) table[i] = pages[i];
    freq[0] = freq[1] = 0.0f; /* no turn: keys arrive as they are */
    paged_append_args_t a = {0};
    a.tokens = a.sequences = B;
    a.type = BMMC_F32;
    a.k = (token_heads_t){k, H, D, H * D, D};
    a.v = (token_heads_t){v, H, D, H * D, D};
    a.turns.inv_freq = freq;
    a.turns.pairs = 2;
    a.lengths = lengths;
    a.table = table;
    a.table_stride = a.table_columns = 2;
    a.pages = PAGES;
    a.page_size = PAGE;
    a.k_cache = (paged_cache_t){kc, PAGE * H * D, H * D, D};
    a.v_cache = (paged_cache_t){vc, PAGE * H * D, H * D, D};
    CHECK(paged_append(&a, NULL));
    if (cudaDeviceSynchronize() != cudaSuccess) return 1;
    const int entry[B] = {4 * PAGE + 0, 2 * PAGE + 3, 0 * PAGE + 1};
    double sum = 0.0;
    for (int i = 0; i < PAGES * PAGE * H * D; ++i) sum += kc[i] + vc[i];
    for (int b = 0; b < B; ++b)
        for (int i = 0; i < H * D; ++i) {
            const float want = (float)(b * H * D + i + 1);
            if (kc[entry[b] * H * D + i] != want || vc[entry[b] * H * D + i] != want) {
                fprintf(stderr, "sequence %d element %d\n", b, i);
                return 1;
            }
            sum -= 2.0 * want;
        }
    return sum == 0.0 ? 0 : 1; /* nothing else was written */
}

int main(void)
{
    int ndev = 0;
    if (cudaGetDeviceCount(&ndev) != cudaSuccess || ndev == 0) {
        printf("no CUDA device\n");
        return 77;
    }
    if (experts() || append()) return 1;
    printf("ok\n");
    return 0;
}

// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   y[i]       = scale * table[tok[i]]
//   dtable[r] (+)= scale * sum of dy[i] over the i with tok[i] = r, i ascending
//
// The sum of a table row is taken in fp32 in an order that depends on the
// tokens alone (positions in order within chunks of the sorted list, chunks in
// order), so that the same inputs give the same bits on every run: no float
// atomics anywhere.
#include "zero_elems.cuh"
#include "zero_ops.h"

namespace zgb {
namespace {

constexpr uint32_t kNone = 0xffffffffu;

// The table row token i names, or -1.
__device__ __forceinline__ int64_t token_row(const TokenArgs &t, int64_t i)
{
    const int64_t id = t.wide ? static_cast<const long long *>(t.ids)[i]
                              : (int64_t)static_cast<const int *>(t.ids)[i];
    return id == t.pad || id < 0 || id >= t.rows ? -1 : id;
}

// ------------------------------------------------------------- the lookup
//
// A warp copies up to 4 x 256 columns of one output row, all in flight at
// once; a wide row takes several warps.  Bound by memory, and for few tokens by
// the two dependent reads (id, row): 131,072 rows of 1600 f16 take 81 us (6.4
// TB/s), 16,384 rows 10 to 13 us, 48 rows of 768 about 2 us on the GPU.  Fewer
// columns in flight are slower (15.2 us with 2 x 256 for 16,384 rows), more
// no faster.
constexpr int kCols = 256;          // columns a warp's lanes hold, 8 each
constexpr int kEmbedFlight = 4;

template <int DT>
__device__ __forceinline__ elems::Span span_of(const void *p, int64_t rows, int64_t stride,
                                               int64_t cols)
{
    // a table without rows has no bytes, whatever its stride (and may be null)
    const char *lo = static_cast<const char *>(p);
    return {lo, rows > 0 ? lo + ((rows - 1) * stride + cols) * elems::Raw<DT>::kSize : lo};
}

template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads)
embed_kernel(const __grid_constant__ EmbedArgs a, int segs)
{
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t task = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int64_t i = task / segs;
    const int seg = (int)(task - i * segs);
    if (i >= a.tok.n) return;
    const int64_t row = token_row(a.tok, i);
    if (row < 0 && a.bad && lane == 0 && seg == 0) {
        const int64_t id = a.tok.wide ? static_cast<const long long *>(a.tok.ids)[i]
                                      : (int64_t)static_cast<const int *>(a.tok.ids)[i];
        // a padding token is no wrong id, but -1 as such stands for none
        if (id != a.tok.pad || id == -1) atomicAdd(a.bad, 1ull);
    }
    const int64_t c0 = (int64_t)seg * kEmbedFlight * kCols;
    const elems::Span table = span_of<DT>(a.table, a.tok.rows, a.table_stride, a.dim);
    const int64_t from = (row >= 0 ? row : 0) * a.table_stride;
    constexpr int kSize = elems::Raw<DT>::kSize;
    const bool inside = table.around((from + c0) * kSize, kEmbedFlight * kCols * kSize);
    elems::Eight<DT, VEC> r[kEmbedFlight];
#pragma unroll
    for (int j = 0; j < kEmbedFlight; ++j) {
        const int64_t c = c0 + j * kCols + lane * 8;
        if constexpr (VEC) {
            r[j].r.zero();
            if (row >= 0 && c < a.dim) r[j].r.load(a.table, from + c);
        } else {
            r[j].ask(a.table, from + c, table, inside);
        }
    }
#pragma unroll
    for (int j = 0; j < kEmbedFlight; ++j) {
        const int64_t first = c0 + j * kCols;
        if (first >= a.dim) break;
        float f[8];
        elems::Raw<DT> w = r[j].take();
        w.get(f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = row >= 0 ? __fmul_rn(f[e], a.scale) : 0.0f;
        w.set(f);
        if (!VEC)
            w.store_any(a.out, i * a.out_stride + first,
                           a.dim - first < kCols ? (int)(a.dim - first) : kCols);
        else if (first + lane * 8 < a.dim)
            w.store(a.out, i * a.out_stride + first + lane * 8);
    }
}

template <int DT, bool VEC> cudaError_t embed_go(const EmbedArgs &a, cudaStream_t s)
{
    const int64_t per = kCols * kEmbedFlight;
    const int64_t segs = (a.dim + per - 1) / per;
    const int64_t warps = a.tok.n * segs;
    // few rows: one warp a block, so that they spread over the SMs (a pass among
    // others shows neither form faster up to 1024 warps, 2.3 to 2.5 us either way;
    // beyond, one warp a block is slower: 2048 rows of 1600 5.0 us against 2.9)
    const int threads = warps <= 1024 ? 32 : kThreads;
    const int64_t blocks = (warps * 32 + threads - 1) / threads;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    return launch_dependent(embed_kernel<DT, VEC>, dim3((unsigned)blocks),
                            dim3((unsigned)threads), 0, s, a, (int)segs);
}

template <int DT> cudaError_t embed_pick(const EmbedArgs &a, cudaStream_t s)
{
    const bool vec = rows_aligned(a.table, a.table_stride, DT, a.dim) &&
                     rows_aligned(a.out, a.out_stride, DT, a.dim);
    return vec ? embed_go<DT, true>(a, s) : embed_go<DT, false>(a, s);
}

// ----------------------------------------------------------------- the sort
//
// (id, position) pairs in order of id, then position; ids that name no row
// come last.  Three ways, by the number of tokens:
//   up to kRankTokens     every token's place is counted outright, as the number of
//                         pairs that come before its own: n^2 comparisons (3 ALU
//                         operations each, 11 us for 8192 tokens), but no
//                         step that waits for another
//   up to kSmallTokens    a stable radix sort by 8-bit digits, lowest first, in one
//                         launch: a cluster of up to 8 blocks with a token a thread,
//                         whose digit counts and tokens go through
//                         distributed shared memory
//   more                  the same over up to 256 blocks, a launch a digit: a block
//                         adds up the digit counts of the blocks before it,
//                         places its tokens, and counts the next digit
//                         where they land
// Up to kFewTokens tokens are not sorted at all (embed_few_kernel).
//
// Where they cross, for the whole gradient into 50,257 rows with ids as
// frequent as a text's, added to fp32 / written as bf16 (us):
//   without a sort or by place   512 x 768: 6.8 / 18.0 or 9.3 / 18.9; 600 x 768: 7.8 /
//                                18.9 or 9.3 / 19.0; 400 x 1600: 7.2 / 30.6 or 9.2 /
//                                35.1; 512 x 1600: 11.7 / 36.9 or 9.3 / 37.9; 1024 x
//                                1600: 19.9 / 51.6 or 9.8 / 43.3
//   by place or by the cluster   1000 x 768: 9.5 / 20.8 or 15.0 / 21.7; 2048 x 768:
//                                12.4 / 25.1 or 15.3 / 22.1; 3000 x 768: 16.4 / 23.8
//                                or 16.1 / 22.8; 8192 x 768: 40.8 / 45.7 or 20.7 / 26.1
constexpr int kSortThreads = 1024, kSortWarps = 32;
constexpr int kFewTokens = 512;
constexpr int kRankTokens = 2048;
constexpr int kSmallTokens = 8192;
constexpr int64_t kSmallRows = 1 << 19;      // id and position in one word
constexpr int kSortTile = 2048;
constexpr int kMaxSortBlocks = 256;

bool sort_small(const EmbedGradArgs &a)
{
    return a.tok.n <= kSmallTokens && a.tok.rows < kSmallRows;
}

int sort_passes(int64_t rows)
{
    int p = 1;
    while (p < 4 && (rows >> (8 * p)) != 0) ++p;   // keys 0 .. rows (rows: names no row)
    return p;
}

int64_t sort_chunk(int64_t n)   // tokens per block of the radix sort
{
    const int64_t per = (n + kMaxSortBlocks - 1) / kMaxSortBlocks;
    return (per + kSortTile - 1) / kSortTile * kSortTile;
}

__device__ __forceinline__ uint32_t token_key(const TokenArgs &t, int64_t i)
{
    const int64_t row = token_row(t, i);
    return row < 0 ? (uint32_t)t.rows : (uint32_t)row;
}

// Lanes of the warp with the same digit (and `live`).
__device__ __forceinline__ uint32_t same_digit(uint32_t d, bool live)
{
    uint32_t m = __ballot_sync(0xffffffffu, live);
#pragma unroll
    for (int b = 0; b < 8; ++b) {
        const uint32_t v = __ballot_sync(0xffffffffu, (d >> b) & 1);
        m &= ((d >> b) & 1) ? v : ~v;
    }
    return m;
}

// Exclusive prefix over the 32 warps of every digit's counts, in place; the
// digits' totals go to total[256].
__device__ __forceinline__ void prefix_warps(unsigned short (*count)[256], uint32_t *total)
{
    for (int d = threadIdx.x; d < 256; d += kSortThreads) {
        uint32_t run = 0;
#pragma unroll 8
        for (int w = 0; w < kSortWarps; ++w) {
            const uint32_t v = count[w][d];
            count[w][d] = (unsigned short)run;
            run += v;
        }
        total[d] = run;
    }
}

// Exclusive prefix of v[256] in place, by the first warp.
__device__ __forceinline__ void prefix_digits(uint32_t *v)
{
    if (threadIdx.x < 32) {
        uint32_t own[8], sum = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            own[j] = v[threadIdx.x * 8 + j];
            sum += own[j];
        }
        uint32_t inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(0xffffffffu, inc, o);
            if ((int)threadIdx.x >= o) inc += u;
        }
        uint32_t run = inc - sum;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[threadIdx.x * 8 + j] = run;
            run += own[j];
        }
    }
}

// A gradient that is not added to has zeros in the rows that no token names.
// All rows are zeroed while the tokens are sorted, which is bound by latency,
// by blocks of the sorts' launches that have no tokens; the sums then write those
// again that a token names.  (A launch of its own that the cluster's sort goes on
// beside: 27.5 us against 25.7 for 8192 tokens of 768 columns.)

// Bytes first .. last of p, 2 KB a warp in turn: this is warp `warp` of `warps`.
__device__ __forceinline__ void zero_bytes(char *p, int64_t first, int64_t last, int64_t warp,
                                           int64_t warps)
{
    const int lane = threadIdx.x & 31;
    const int64_t rest = (16 - (int64_t)((uintptr_t)(p + first) & 15)) & 15;
    const int64_t head = first + rest < last ? first + rest : last;
    const int64_t whole = (last - head) / 16, tail = head + whole * 16;
    const uint4 z = make_uint4(0, 0, 0, 0);
    uint4 *v = reinterpret_cast<uint4 *>(p + head);
    for (int64_t i = warp * 128 + lane; i < whole; i += warps * 128) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (i + u * 32 < whole) v[i + u * 32] = z;
    }
    if (warp != 0) return;
    if (lane < head - first) p[first + lane] = 0;
    if (lane < last - tail) p[tail + lane] = 0;
}

// Rows lo .. hi: this is warp `warp` of `warps`.  Rows that follow one another
// are one piece of memory; blocks of 32 warps write aligned ones faster row by
// row (50,257 x 1600 16-bit zeroes beside 16,384 tokens' sort: 52 us against
// 54.6), blocks of 8 not (30.6 us as a piece, 34.5 by rows).
template <int GT, bool VEC>
__device__ __forceinline__ void zero_rows(const EmbedGradArgs &a, int64_t lo, int64_t hi,
                                          int64_t warp, int64_t warps)
{
    constexpr int kSize = elems::Raw<GT>::kSize;
    if (a.grad_stride == a.dim && (!VEC || blockDim.x == kThreads)) {
        zero_bytes(static_cast<char *>(a.grad), lo * a.dim * kSize, hi * a.dim * kSize,
                   warp, warps);
        return;
    }
    elems::Raw<GT> z;
    z.zero();
    for (int64_t r = lo + warp; r < hi; r += warps)
        for (int64_t c = 0; c < a.dim; c += kCols) {
            const int64_t at = r * a.grad_stride + c;
            if (!VEC) z.store_any(a.grad, at, a.dim - c < kCols ? (int)(a.dim - c) : kCols);
            else if (c + (threadIdx.x & 31) * 8 < a.dim) z.store(a.grad, at + (threadIdx.x & 31) * 8);
        }
}

// The first rank_blocks blocks place 32 tokens each, one a lane, each warp against
// an eighth of the list, which it reads from shared memory four pairs at a
// time, the same for all lanes.  The others zero rows.
template <int GT, bool VEC>
__global__ void __launch_bounds__(kThreads)
embed_rank_kernel(const __grid_constant__ EmbedGradArgs a, int rank_blocks)
{
    __shared__ __align__(16) uint32_t pairs[kRankTokens];
    __shared__ uint32_t part[8][32];
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if ((int)blockIdx.x >= rank_blocks) {
        zero_rows<GT, VEC>(a, 0, a.tok.rows, (int64_t)(blockIdx.x - rank_blocks) * 8 + warp,
                           (int64_t)(gridDim.x - rank_blocks) * 8);
        return;
    }
    const int n = (int)a.tok.n;
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.n_runs = 0;
    // eight warps' whole rounds of 16, the last filled up with what comes after all
    const int padded = (n + 127) / 128 * 128;
    uint32_t k[kRankTokens / kThreads];
#pragma unroll
    for (int u = 0; u < kRankTokens / kThreads; ++u) {
        const int i = (int)threadIdx.x + u * kThreads;
        k[u] = i < n ? token_key(a.tok, i) << 13 | (uint32_t)i : kNone;
    }
#pragma unroll
    for (int u = 0; u < kRankTokens / kThreads; ++u) pairs[threadIdx.x + u * kThreads] = k[u];
    __syncthreads();
    const int i = (int)blockIdx.x * 32 + lane;
    const uint32_t own = i < n ? pairs[i] : 0u;
    uint32_t before = 0;
    const uint4 *v = reinterpret_cast<const uint4 *>(pairs) + warp * (padded / 32);
    for (int j = 0; j < padded / 128; ++j, v += 4) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const uint4 p = v[u];
            before += (p.x < own) + (p.y < own) + (p.z < own) + (p.w < own);
        }
    }
    part[warp][lane] = before;
    __syncthreads();
    if (warp == 0 && i < n) {
        uint32_t at = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) at += part[w][lane];
        a.key[0][at] = own >> 13;
        a.idx[0][at] = (uint32_t)i;
    }
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_arrive()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}

__device__ __forceinline__ void cluster_wait()
{
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void cluster_sync()
{
    cluster_arrive();
    cluster_wait();
}

__device__ __forceinline__ void store_peer(const void *p, uint32_t rank, uint32_t v)
{
    uint32_t at;
    asm("mapa.shared::cluster.u32 %0, %1, %2;"
        : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

// The first cluster sorts, the others zero rows.  A pair is one word (id << 13
// | position), a thread has one in every pass.
template <int GT, bool VEC>
__global__ void __launch_bounds__(kSortThreads)
embed_cluster_kernel(const __grid_constant__ EmbedGradArgs a, int passes, int blocks)
{
    __shared__ uint32_t list[2][kSortThreads];
    __shared__ unsigned short count[kSortWarps][256];
    __shared__ uint32_t total[256], hist[8][256], sum[256], before[256];
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if ((int)blockIdx.x >= blocks) {
        zero_rows<GT, VEC>(a, 0, a.tok.rows,
                           (int64_t)(blockIdx.x - blocks) * kSortWarps + warp,
                           (int64_t)(gridDim.x - blocks) * kSortWarps);
        return;
    }
    // A block's shared memory may be written to once it is known to run: each
    // arrives here, and waits for the others before its first store to them.
    cluster_arrive();
    const uint32_t rank = cluster_rank();
    const int n = (int)a.tok.n, i = (int)rank * kSortThreads + (int)threadIdx.x;
    const bool live = i < n;                  // the places 0 .. n are taken in every pass
    if (i == 0) *a.n_runs = 0;
    list[0][threadIdx.x] = live ? token_key(a.tok, i) << 13 | (uint32_t)i : kNone;
    for (int p = 0; p < passes; ++p) {
        for (int c = threadIdx.x; c < kSortWarps * 128; c += kSortThreads)
            reinterpret_cast<uint32_t *>(&count[0][0])[c] = 0;
        __syncthreads();
        const uint32_t pair = list[p & 1][threadIdx.x], d = (pair >> (13 + 8 * p)) & 255u;
        const uint32_t peers = same_digit(d, live);
        if (live && (peers >> lane) == 1u) count[warp][d] = (unsigned short)__popc(peers);
        __syncthreads();
        prefix_warps(count, total);
        __syncthreads();
        if (p == 0) cluster_wait();
        // every block gets every block's counts
        for (int c = threadIdx.x; c < 256 * blocks; c += kSortThreads)
            store_peer(&hist[rank][c & 255], (uint32_t)c >> 8, total[c & 255]);
        cluster_sync();
        if (threadIdx.x < 256) {
            uint32_t all = 0, mine = 0;
            for (int q = 0; q < blocks; ++q) {
                const uint32_t v = hist[q][threadIdx.x];
                all += v;
                mine += q < (int)rank ? v : 0u;
            }
            sum[threadIdx.x] = all;
            before[threadIdx.x] = mine;
        }
        __syncthreads();
        prefix_digits(sum);
        __syncthreads();
        if (live) {
            const uint32_t at = sum[d] + before[d] + count[warp][d] +
                                __popc(peers & ((1u << lane) - 1));
            store_peer(&list[(p & 1) ^ 1][at & (kSortThreads - 1)], at / kSortThreads, pair);
        }
        cluster_sync();
    }
    if (live) {
        const uint32_t pair = list[passes & 1][threadIdx.x];
        a.key[0][i] = pair >> 13;
        a.idx[0][i] = pair & 8191u;
    }
}

// Counts of the first digit, a block at a time.  The later digits' counts and
// the count of long runs are cleared here; the blocks past sort_blocks zero rows.
template <int GT, bool VEC>
__global__ void __launch_bounds__(kSortThreads)
embed_count_kernel(const __grid_constant__ EmbedGradArgs a, int64_t chunk, int passes,
                   int sort_blocks)
{
    __shared__ uint32_t count[256];
    pdl_wait();
    pdl_launch_dependents();
    if ((int)blockIdx.x >= sort_blocks) {
        zero_rows<GT, VEC>(a, 0, a.tok.rows / (passes + 1),
                           (int64_t)(blockIdx.x - sort_blocks) * kSortWarps + (threadIdx.x >> 5),
                           (int64_t)(gridDim.x - sort_blocks) * kSortWarps);
        return;
    }
    const int64_t T = (int64_t)sort_blocks * kSortThreads;
    const int64_t t0 = (int64_t)blockIdx.x * kSortThreads + threadIdx.x;
    if (t0 == 0) *a.n_runs = 0;
    for (int64_t i = t0; i < (int64_t)(passes - 1) * sort_blocks * 256; i += T)
        a.hist[(int64_t)sort_blocks * 256 + i] = 0;
    if (threadIdx.x < 256) count[threadIdx.x] = 0;
    __syncthreads();
    const int64_t lo = (int64_t)blockIdx.x * chunk;
    const int64_t hi = lo + chunk < a.tok.n ? lo + chunk : a.tok.n;
#pragma unroll 2
    for (int64_t i = lo + threadIdx.x; i < hi; i += kSortThreads)
        atomicAdd(&count[token_key(a.tok, i) & 255u], 1u);
    __syncthreads();
    if (threadIdx.x < 256) a.hist[blockIdx.x * 256 + threadIdx.x] = count[threadIdx.x];
}

// Pass `pass` reads side (pass & 1) ^ 1 (the tokens themselves at first) and
// writes side pass & 1.  The blocks past sort_blocks zero rows.
template <int GT, bool VEC>
__global__ void __launch_bounds__(kSortThreads)
embed_place_kernel(const __grid_constant__ EmbedGradArgs a, int pass, int passes, int64_t chunk,
                   int sort_blocks)
{
    __shared__ unsigned short count[kSortWarps][256];
    __shared__ uint32_t total[256], base[256], local[256], part[4][2][256];
    __shared__ uint32_t tile_key[kSortTile], tile_idx[kSortTile];
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if ((int)blockIdx.x >= sort_blocks) {
        zero_rows<GT, VEC>(a, a.tok.rows * (pass + 1) / (passes + 1),
                         a.tok.rows * (pass + 2) / (passes + 1),
                         (int64_t)(blockIdx.x - sort_blocks) * kSortWarps + warp,
                         (int64_t)(gridDim.x - sort_blocks) * kSortWarps);
        return;
    }
    const uint32_t *hist = a.hist + (int64_t)pass * sort_blocks * 256;
    uint32_t *next = pass + 1 < passes ? a.hist + (int64_t)(pass + 1) * sort_blocks * 256 : nullptr;
    {   // tokens of each digit in all blocks, and in the blocks before this one
        const int d = threadIdx.x & 255, quarter = threadIdx.x >> 8;
        uint32_t all = 0, before = 0;
#pragma unroll 8
        for (int b = quarter; b < sort_blocks; b += 4) {
            const uint32_t v = hist[b * 256 + d];
            all += v;
            before += b < (int)blockIdx.x ? v : 0u;
        }
        part[quarter][0][d] = all;
        part[quarter][1][d] = before;
    }
    __syncthreads();
    if (threadIdx.x < 256)
        total[threadIdx.x] = part[0][0][threadIdx.x] + part[1][0][threadIdx.x] +
                             part[2][0][threadIdx.x] + part[3][0][threadIdx.x];
    __syncthreads();
    prefix_digits(total);
    __syncthreads();
    if (threadIdx.x < 256)
        base[threadIdx.x] = total[threadIdx.x] + part[0][1][threadIdx.x] +
                            part[1][1][threadIdx.x] + part[2][1][threadIdx.x] +
                            part[3][1][threadIdx.x];
    const uint32_t *skey = a.key[(pass & 1) ^ 1], *sidx = a.idx[(pass & 1) ^ 1];
    uint32_t *dkey = a.key[pass & 1], *didx = a.idx[pass & 1];
    const int64_t lo = (int64_t)blockIdx.x * chunk;
    const int64_t hi = lo + chunk < a.tok.n ? lo + chunk : a.tok.n;
    constexpr int kIters = kSortTile / kSortThreads;
    for (int64_t tile = lo; tile < hi; tile += kSortTile) {
        for (int i = threadIdx.x; i < kSortWarps * 128; i += kSortThreads)
            reinterpret_cast<uint32_t *>(&count[0][0])[i] = 0;
        __syncthreads();
        uint32_t key[kIters], idx[kIters], rank[kIters];
#pragma unroll
        for (int j = 0; j < kIters; ++j) {
            const int64_t i = tile + (warp * kIters + j) * 32 + lane;
            const bool live = i < hi;
            key[j] = !live ? kNone : pass == 0 ? token_key(a.tok, i) : skey[i];
            idx[j] = !live ? 0u : pass == 0 ? (uint32_t)i : sidx[i];
        }
#pragma unroll
        for (int j = 0; j < kIters; ++j) {
            const bool live = tile + (warp * kIters + j) * 32 + lane < hi;
            const uint32_t d = (key[j] >> (8 * pass)) & 255u;
            const uint32_t peers = same_digit(d, live);
            uint32_t before = 0;
            if (live) before = count[warp][d];
            __syncwarp();
            rank[j] = before + __popc(peers & ((1u << lane) - 1));
            if (live && (peers >> lane) == 1u)
                count[warp][d] = (unsigned short)(before + __popc(peers));
            __syncwarp();
        }
        __syncthreads();
        prefix_warps(count, total);
        __syncthreads();
        if (threadIdx.x < 256) local[threadIdx.x] = total[threadIdx.x];
        __syncthreads();
        prefix_digits(local);
        __syncthreads();
        // in order within the block first, so that neighbouring threads then write
        // neighbouring places
#pragma unroll
        for (int j = 0; j < kIters; ++j)
            if (tile + (warp * kIters + j) * 32 + lane < hi) {
                const uint32_t d = (key[j] >> (8 * pass)) & 255u;
                const uint32_t at = local[d] + count[warp][d] + rank[j];
                tile_key[at] = key[j];
                tile_idx[at] = idx[j];
            }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kIters; ++j) {
            const int i = j * kSortThreads + (int)threadIdx.x;
            const bool live = tile + i < hi;
            uint32_t cell = kNone;
            if (live) {
                const uint32_t k = tile_key[i], d = (k >> (8 * pass)) & 255u;
                const uint32_t at = base[d] - local[d] + (uint32_t)i;
                dkey[at] = k;
                didx[at] = tile_idx[i];
                cell = at / (uint32_t)chunk * 256 + ((k >> (8 * pass + 8)) & 255u);
            }
            if (next) {     // one addition for a warp's tokens of one cell: a frequent id has many
                const uint32_t peers = __match_any_sync(0xffffffffu, cell);
                if (live && (peers >> lane) == 1u) atomicAdd(&next[cell], (uint32_t)__popc(peers));
            }
        }
        __syncthreads();
        if (threadIdx.x < 256) base[threadIdx.x] += total[threadIdx.x];
    }
}

// ------------------------------------------------------------------ the sums
//
// The sorted list is cut into chunks of C positions.  A warp takes a chunk
// and 256 columns, 8 a lane, and reads the chunk's rows of dy a few at a
// time.  A run of one id that lies within the chunk is finished there.  One that
// passes an end of it leaves its fp32 part in the workspace (slot 0: the run
// that the chunk begins in the middle of, slot 1: the run that passes its end),
// and the chunk in which such a run begins enters it in a list whose entries
// embed_runs_kernel finishes.  The rows of dy bound it: 131,071 of 1600 f16
// columns with ids as frequent as a text's take 82 us (420 MB read, 6.2 TB/s with
// the writes), the list's runs 13.  (Counting the parts, for whichever warp brings
// the last one to add them up in the same launch, costs a fence a part: 207 us
// against 103 for 131,071 tokens of 1600 columns.)
int64_t sum_chunk(int64_t n)
{
    int64_t c = n <= kRankTokens ? 8 : 16;
    while (c < 256 && n > c * 2048) c *= 2;
    return c;
}

// The 256 columns from c0 of a row of the gradient, as they are before.
template <int GT, bool VEC>
__device__ __forceinline__ void ask_row(const EmbedGradArgs &a, const elems::Span &grad,
                                        uint32_t row, int64_t c0, elems::Eight<GT, VEC> &r)
{
    constexpr int kSize = elems::Raw<GT>::kSize;
    const int64_t c = c0 + (threadIdx.x & 31) * 8, from = (int64_t)row * a.grad_stride;
    r.ask(a.grad, from + (VEC && c >= a.dim ? a.dim - 8 : c), grad,
          grad.around((from + c0) * kSize, kCols * kSize));
}

// By the whole warp: the sums of 256 columns from c0 go to a row of the
// gradient; ACC: are added to `old`.
template <int GT, bool VEC, bool ACC>
__device__ __forceinline__ void put_row(const EmbedGradArgs &a, uint32_t row, int64_t c0,
                                        const float (&acc)[8], const elems::Raw<GT> &old)
{
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = __fmul_rn(acc[e], a.scale);
    if (ACC) {
        float o[8];
        old.get(o);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = __fadd_rn(o[e], f[e]);
    }
    elems::Raw<GT> r;
    r.set(f);
    const int64_t at = (int64_t)row * a.grad_stride + c0;
    if (!VEC) r.store_any(a.grad, at, a.dim - c0 < kCols ? (int)(a.dim - c0) : kCols);
    else if (c0 + (threadIdx.x & 31) * 8 < a.dim) r.store(a.grad, at + (threadIdx.x & 31) * 8);
}

__device__ __forceinline__ void put_part(float *p, const float (&acc)[8])
{
    reinterpret_cast<float4 *>(p)[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
}

// Up to kFewTokens tokens, without a sort: a block takes a token, and ends at
// once if an earlier one has its id.  Otherwise it lists the positions of that
// id and adds up their rows, a warp 256 columns; of a narrow table, and of an
// id with many positions, several warps share the columns and take the positions
// in turn, and their sums join in the warps' order.  Without ACC the blocks past
// the tokens' zero the rows that no token names, a slice of the table each: they
// mark the named rows of kMarkRows rows at a time and write what lies between
// them, so that no row is written twice and one launch does (512 tokens into
// 50,257 x 768 bf16: 13.3 us, against 24.4 with the zeroes in a launch before).
constexpr int kMarkRows = 8192;

template <int GT, bool VEC>
__device__ __forceinline__ void zero_unnamed(const EmbedGradArgs &a, int64_t slice, int64_t slices)
{
    __shared__ uint32_t mark[kMarkRows / 32];
    static_assert(kMarkRows / 32 == kThreads, "a word a thread");
    const int warp = threadIdx.x >> 5;
    int64_t row[kFewTokens / kThreads];
#pragma unroll
    for (int u = 0; u < kFewTokens / kThreads; ++u) {
        const int j = u * kThreads + (int)threadIdx.x;
        row[u] = j < (int)a.tok.n ? token_row(a.tok, j) : -1;
    }
    const int64_t end = a.tok.rows * (slice + 1) / slices;
    for (int64_t lo = a.tok.rows * slice / slices; lo < end; lo += kMarkRows) {
        const int m = (int)(end - lo < kMarkRows ? end - lo : kMarkRows);
        __syncthreads();
        mark[threadIdx.x] = 0;
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kFewTokens / kThreads; ++u)
            if (row[u] >= lo && row[u] < lo + m)
                atomicOr(&mark[(row[u] - lo) >> 5], 1u << ((row[u] - lo) & 31));
        __syncthreads();
        for (int r = 0; r < m;) {
            // the next named row from r on, the same for every thread
            int w = r >> 5;
            uint32_t bits = mark[w] & (0xffffffffu << (r & 31));
            while (!bits && (w + 1) * 32 < m) bits = mark[++w];
            const int next = bits ? w * 32 + __ffs(bits) - 1 : m;
            if (next > r) zero_rows<GT, VEC>(a, lo + r, lo + next, warp, kThreads / 32);
            r = next + 1;
        }
    }
}

template <int YT, int GT, bool VEC, bool ACC>
__global__ void __launch_bounds__(kThreads)
embed_few_kernel(const __grid_constant__ EmbedGradArgs a, int segs, int least)
{
    constexpr int U = YT == F32 || !VEC ? 4 : 8;
    __shared__ unsigned short list[kFewTokens];
    __shared__ uint32_t found[kFewTokens / 32];
    __shared__ int n_list;
    __shared__ float sums[8][kCols];
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n = (int)a.tok.n, i = (int)blockIdx.x;
    if (!ACC && i >= n) {
        zero_unnamed<GT, VEC>(a, i - n, (int64_t)gridDim.x - n);
        return;
    }
    const int64_t id = token_row(a.tok, i);
    bool again = false;
    if (id >= 0) {
        int64_t other[kFewTokens / kThreads];
#pragma unroll
        for (int u = 0; u < kFewTokens / kThreads; ++u) {
            const int j = u * kThreads + (int)threadIdx.x;
            other[u] = j < n ? token_row(a.tok, j) : -1;
        }
#pragma unroll
        for (int u = 0; u < kFewTokens / kThreads; ++u) {
            const int j = u * kThreads + (int)threadIdx.x;
            again |= other[u] == id && j < i;
            const uint32_t m = __ballot_sync(0xffffffffu, other[u] == id);
            if (lane == 0) found[u * 8 + warp] = m;
        }
    }
    // nothing to do (the same for the whole block)
    const bool idle = __syncthreads_or(again) || id < 0;
    if (!idle) {
        if (warp == 0) {
            static_assert(kFewTokens % 64 == 0 && kFewTokens <= 2048, "two words a lane");
            const bool has = lane < kFewTokens / 64;
            const uint32_t m0 = has ? found[2 * lane] : 0u, m1 = has ? found[2 * lane + 1] : 0u;
            const int own = __popc(m0) + __popc(m1);
            int at = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, at, o);
                if (lane >= o) at += v;
            }
            if (lane == 31) n_list = at;
            at -= own;
            for (uint32_t m = m0; m; m &= m - 1)
                list[at++] = (unsigned short)(lane * 64 + __ffs(m) - 1);
            for (uint32_t m = m1; m; m &= m - 1)
                list[at++] = (unsigned short)(lane * 64 + 32 + __ffs(m) - 1);
        }
        __syncthreads();
        const int count = n_list, shares = count > 32 ? 8 : least;
        const int share = warp % shares, lead = warp / shares * shares;
        const elems::Span dy = span_of<YT>(a.dy, a.tok.n, a.dy_stride, a.dim);
        const elems::Span grad = span_of<GT>(a.grad, a.tok.rows, a.grad_stride, a.dim);
        constexpr int kSize = elems::Raw<YT>::kSize;
        // the same number of rounds for every warp: they join through shared memory
        for (int seg0 = 0; seg0 < segs; seg0 += 8 / shares) {
            const int seg = seg0 + warp / shares;
            const int64_t c0 = (int64_t)seg * kCols;
            const int64_t col = c0 + lane * 8 < a.dim || !VEC ? c0 + lane * 8 : a.dim - 8;
            elems::Eight<GT, VEC> old;
            float acc[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
            if (seg < segs) {
                if (ACC && share == 0) ask_row<GT, VEC>(a, grad, (uint32_t)id, c0, old);
                for (int k = share; k < count; k += U * shares) {
                    elems::Eight<YT, VEC> r[U];
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int64_t p = list[k + u * shares < count ? k + u * shares : k];
                        r[u].ask(a.dy, p * a.dy_stride + col, dy,
                                 dy.around((p * a.dy_stride + c0) * kSize, kCols * kSize));
                    }
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        if (k + u * shares >= count) break;
                        float f[8];
                        r[u].take().get(f);
#pragma unroll
                        for (int e = 0; e < 8; ++e) acc[e] = __fadd_rn(acc[e], f[e]);
                    }
                }
            }
            if (shares > 1 && count > 1) {
#pragma unroll
                for (int e = 0; e < 8; ++e) sums[warp][lane * 8 + e] = acc[e];
                __syncthreads();
                if (share == 0) {
                    for (int w = 1; w < shares && w < count; ++w)
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            acc[e] = __fadd_rn(acc[e], sums[lead + w][lane * 8 + e]);
                }
                __syncthreads();
            }
            if (seg < segs && share == 0) {
                elems::Raw<GT> was;
                if (ACC) was = old.take();
                put_row<GT, VEC, ACC>(a, (uint32_t)id, c0, acc, was);
            }
        }
    }
}

template <int YT, int GT, bool VEC, bool ACC>
__global__ void __launch_bounds__(kThreads)
embed_sum_kernel(const __grid_constant__ EmbedGradArgs a, int side, int64_t chunk, int segs)
{
    constexpr int U = YT == F32 || ACC || !VEC ? 4 : 8;       // rows in flight
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t task = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int64_t ck = task / segs;
    const int seg = (int)(task - ck * segs);
    const int64_t lo = ck * chunk;
    if (lo >= a.tok.n) return;
    const int64_t hi = lo + chunk < a.tok.n ? lo + chunk : a.tok.n;
    const uint32_t *key = a.key[side], *idx = a.idx[side];
    const uint32_t none = (uint32_t)a.tok.rows;
    uint32_t mykey = none, myidx = 0;             // of position base + lane, base = lo at first
    if (lo + lane < hi) {
        mykey = key[lo + lane];
        myidx = idx[lo + lane];
    }
    uint32_t edge = kNone;                        // the ids around the chunk
    if (lane == 0 && lo > 0) edge = key[lo - 1];
    if (lane == 1 && hi < a.tok.n) edge = key[hi];
    const uint32_t prev = __shfl_sync(0xffffffffu, edge, 0);
    const uint32_t next = __shfl_sync(0xffffffffu, edge, 1);
    const uint32_t first = __shfl_sync(0xffffffffu, mykey, 0);
    if (first == none) return;                    // sorted: nothing but such ids follows
    const elems::Span dy = span_of<YT>(a.dy, a.tok.n, a.dy_stride, a.dim);
    const elems::Span grad = span_of<GT>(a.grad, a.tok.rows, a.grad_stride, a.dim);
    constexpr int kSize = elems::Raw<YT>::kSize;
    const int64_t c0 = (int64_t)seg * kCols;
    // a lane past the row's end reads its last columns again (VEC), or what
    // lies behind them in the matrix (ANY): neither is written
    const int64_t col = c0 + lane * 8 < a.dim || !VEC ? c0 + lane * 8 : a.dim - 8;
    float *part = a.part + ck * 2 * (int64_t)segs * kCols + c0 + lane * 8;
    bool begun = prev != first;                   // the current run began in this chunk
    bool open = false;                            // and has not ended
    float acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.0f;

    for (int64_t base = lo; base < hi; base += 32) {
        const int m = (int)(hi - base < 32 ? hi - base : 32);
        if (base > lo) {
            mykey = lane < m ? key[base + lane] : none;
            myidx = lane < m ? idx[base + lane] : 0u;
        }
        // which positions have a row, and which of them end their run
        uint32_t after = __shfl_down_sync(0xffffffffu, mykey, 1);
        if (lane == m - 1) after = base + m < hi ? key[base + m] : next;
        const uint32_t live = __ballot_sync(0xffffffffu, lane < m && mykey != none);
        const uint32_t ends = __ballot_sync(0xffffffffu, after != mykey) & live;
        for (int u0 = 0; u0 < m; u0 += U) {
            // every lane loads, whatever of it is used: position 0 stands in for
            // what is not there
            elems::Eight<YT, VEC> r[U];
            elems::Eight<GT, VEC> old[ACC ? U : 1];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t i = __shfl_sync(0xffffffffu, myidx, u0 + u);
                r[u].ask(a.dy, i * a.dy_stride + col, dy,
                         dy.around((i * a.dy_stride + c0) * kSize, kCols * kSize));
            }
            if constexpr (ACC) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const uint32_t k = __shfl_sync(0xffffffffu, mykey, u0 + u);
                    if (ends >> (u0 + u) & 1) ask_row<GT, VEC>(a, grad, k, c0, old[u]);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (!(live >> (u0 + u) & 1)) break;
                float f[8];
                r[u].take().get(f);
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] = __fadd_rn(acc[e], f[e]);
                open = true;
                if (!(ends >> (u0 + u) & 1)) continue;
                if (begun) {
                    elems::Raw<GT> was;
                    if (ACC) was = old[ACC ? u : 0].take();
                    put_row<GT, VEC, ACC>(a, __shfl_sync(0xffffffffu, mykey, u0 + u), c0, acc, was);
                } else {
                    put_part(part, acc);
                }
                begun = true;
                open = false;
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
            }
        }
    }
    if (!open) return;
    put_part(part + (begun ? (int64_t)segs * kCols : 0), acc);
    if (begun && seg == 0 && lane == 0) a.runs[atomicAdd(a.n_runs, 1u)] = (uint32_t)ck;
}

// Adds the parts of chunks from, from + step, ... up to `last` to acc; chunk
// `first` has its part in the second slot.
__device__ __forceinline__ void add_parts(const float *p0, int64_t width, int64_t slot,
                                          int64_t from, int64_t last, int64_t step,
                                          int64_t first, float (&acc)[8])
{
#pragma unroll 4
    for (int64_t c = from; c <= last; c += step) {
        const float *p = p0 + c * width + (c == first ? slot : 0);
        const float4 u = reinterpret_cast<const float4 *>(p)[0];
        const float4 v = reinterpret_cast<const float4 *>(p)[1];
        acc[0] = __fadd_rn(acc[0], u.x);
        acc[1] = __fadd_rn(acc[1], u.y);
        acc[2] = __fadd_rn(acc[2], u.z);
        acc[3] = __fadd_rn(acc[3], u.w);
        acc[4] = __fadd_rn(acc[4], v.x);
        acc[5] = __fadd_rn(acc[5], v.y);
        acc[6] = __fadd_rn(acc[6], v.z);
        acc[7] = __fadd_rn(acc[7], v.w);
    }
}

// A warp takes a listed run and 256 columns and adds up its chunks' parts in
// their order.  Runs of more than kLongRun parts it leaves to its block, whose
// warps then take every eighth part each; their eight sums join in the warps'
// order.  Neighbouring tasks (a run's columns) go to different blocks, so that a
// frequent id does not keep one block busy.  (131,071 tokens x 1600 f16: 133 us
// with 24 parts as with 8, 140 with 96.)
constexpr int kLongRun = 24, kLongMost = 64;

template <int GT, bool VEC, bool ACC>
__global__ void __launch_bounds__(kThreads)
embed_runs_kernel(const __grid_constant__ EmbedGradArgs a, int side, int64_t chunk, int segs)
{
    __shared__ float sums[8][kCols];
    __shared__ int64_t long_first[kLongMost], long_last[kLongMost];
    __shared__ int long_seg[kLongMost], n_long;
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t tasks = (int64_t)*a.n_runs * segs;
    const uint32_t *key = a.key[side];
    const int64_t width = 2 * (int64_t)segs * kCols, slot = (int64_t)segs * kCols;
    const elems::Span grad = span_of<GT>(a.grad, a.tok.rows, a.grad_stride, a.dim);
    if (threadIdx.x == 0) n_long = 0;
    __syncthreads();
    for (int64_t t = blockIdx.x + (int64_t)gridDim.x * warp; t < tasks;
         t += (int64_t)gridDim.x * 8) {
        const int64_t run = t / segs;
        const int seg = (int)(t - run * segs);
        const int64_t first = a.runs[run];
        // the last chunk whose first id is the run's: 32 chunks at a time
        uint32_t id = 0;
        int64_t last = first;
        for (int64_t c = first + 1;; c += 32) {
            const int64_t at = (c + lane) * chunk;
            const uint32_t k = at < a.tok.n ? key[at] : kNone;
            if (c == first + 1) id = __shfl_sync(0xffffffffu, k, 0);
            const uint32_t m = __ballot_sync(0xffffffffu, k == id);
            last = c + (m == 0xffffffffu ? 31 : __ffs(~m) - 2);
            if (m != 0xffffffffu) break;
        }
        const float *p0 = a.part + (int64_t)seg * kCols + lane * 8;
        const bool is_long = last - first >= kLongRun;
        if (is_long) {
            int at = kLongMost;
            if (lane == 0) at = atomicAdd(&n_long, 1);
            at = __shfl_sync(0xffffffffu, at, 0);
            if (at < kLongMost) {
                if (lane == 0) {
                    long_first[at] = first;
                    long_last[at] = last;
                    long_seg[at] = seg;
                }
                continue;
            }
        }
        elems::Eight<GT, VEC> old;
        if (ACC) ask_row<GT, VEC>(a, grad, id, (int64_t)seg * kCols, old);
        float acc[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
        if (!is_long) {
            add_parts(p0, width, slot, first, last, 1, first, acc);
        } else {     // the block's list is full: the same sums, one after another
            for (int w = 0; w < 8; ++w) {
                float part[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) part[e] = 0.0f;
                add_parts(p0, width, slot, first + w, last, 8, first, part);
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] = w ? __fadd_rn(acc[e], part[e]) : part[e];
            }
        }
        elems::Raw<GT> was;
        if (ACC) was = old.take();
        put_row<GT, VEC, ACC>(a, id, (int64_t)seg * kCols, acc, was);
    }
    __syncthreads();
    const int count = n_long < kLongMost ? n_long : kLongMost;
    for (int i = 0; i < count; ++i) {
        const int64_t first = long_first[i], last = long_last[i];
        const int seg = long_seg[i];
        float acc[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
        add_parts(a.part + (int64_t)seg * kCols + lane * 8, width, slot, first + warp, last, 8,
                  first, acc);
#pragma unroll
        for (int e = 0; e < 8; ++e) sums[warp][lane * 8 + e] = acc[e];
        __syncthreads();
        if (warp == 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float s = sums[0][lane * 8 + e];
#pragma unroll
                for (int w = 1; w < 8; ++w) s = __fadd_rn(s, sums[w][lane * 8 + e]);
                acc[e] = s;
            }
            const uint32_t id = key[(first + 1) * chunk];
            elems::Eight<GT, VEC> old;
            elems::Raw<GT> was;
            if (ACC) {
                ask_row<GT, VEC>(a, grad, id, (int64_t)seg * kCols, old);
                was = old.take();
            }
            put_row<GT, VEC, ACC>(a, id, (int64_t)seg * kCols, acc, was);
        }
        __syncthreads();
    }
}

template <int GT, bool VEC>
cudaError_t small_go(const EmbedGradArgs &a, int sms, cudaStream_t s)
{
    if (a.tok.n <= kRankTokens) {
        const int blocks = (int)((a.tok.n + 31) / 32), fill = a.accumulate ? 0 : 4 * sms;
        return launch_dependent(embed_rank_kernel<GT, VEC>, dim3((unsigned)(blocks + fill)),
                                dim3(kThreads), 0, s, a, blocks);
    }
    int blocks = 1;
    while (blocks * kSortThreads < a.tok.n) blocks *= 2;
    const int fill = a.accumulate ? 0 : 2 * sms / blocks * blocks;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(blocks + fill));
    cfg.blockDim = dim3(kSortThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)blocks;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, embed_cluster_kernel<GT, VEC>, a, sort_passes(a.tok.rows),
                              blocks);
}

template <int YT, int GT, bool VEC, bool ACC>
cudaError_t grad_go(const EmbedGradArgs &a, int sms, cudaStream_t s)
{
    const int64_t n = a.tok.n;
    const int segs = (int)((a.dim + kCols - 1) / kCols);
    int side = 0;
    cudaError_t e;
    if (n <= kFewTokens) {
        const int least = segs == 1 ? 8 : segs == 2 ? 4 : segs <= 4 ? 2 : 1;
        // zeroes: 32 KB a block, within 1 and 16 blocks an SM (4 for any table: 14.9
        // us for the 77 MB above, 4.2 for 128 KB, against 13.3 and 3.6)
        const int64_t room = a.tok.rows * a.dim * elem_size(GT) >> 15, most = 16 * (int64_t)sms;
        const int64_t fill = ACC ? 0 : room < sms ? sms : room < most ? room : most;
        return launch_dependent(embed_few_kernel<YT, GT, VEC, ACC>, dim3((unsigned)(n + fill)),
                                dim3(kThreads), 0, s, a, segs, least);
    }
    if (sort_small(a)) {
        e = small_go<GT, VEC>(a, sms, s);
        if (e != cudaSuccess) return e;
    } else {
        const int passes = sort_passes(a.tok.rows);
        const int64_t chunk = sort_chunk(n);
        const int blocks = (int)((n + chunk - 1) / chunk);
        const int fill = ACC ? 0 : 2 * sms;
        e = launch_dependent(embed_count_kernel<GT, VEC>, dim3((unsigned)(blocks + fill)),
                             dim3(kSortThreads), 0, s, a, chunk, passes, blocks);
        if (e != cudaSuccess) return e;
        for (int p = 0; p < passes; ++p) {
            e = launch_dependent(embed_place_kernel<GT, VEC>, dim3((unsigned)(blocks + fill)),
                                 dim3(kSortThreads), 0, s, a, p, passes, chunk, blocks);
            if (e != cudaSuccess) return e;
        }
        side = (passes - 1) & 1;
    }
    const int64_t chunk = sum_chunk(n);
    const int64_t tasks = (n + chunk - 1) / chunk * segs;
    // few tasks spread over the SMs (2048 tokens of 768: 12.4 us against 12.9 with
    // 8 warps a block; for many there is nothing in it, 34.3 against 35.4 at 16,384)
    const int threads = tasks <= 16 * (int64_t)sms ? 64 : kThreads;
    const int64_t blocks = (tasks * 32 + threads - 1) / threads;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    e = launch_dependent(embed_sum_kernel<YT, GT, VEC, ACC>, dim3((unsigned)blocks),
                         dim3((unsigned)threads), 0, s, a, side, chunk, segs);
    if (e != cudaSuccess) return e;
    const int64_t most = (tasks + 7) / 8, grid = most < 8 * (int64_t)sms ? most : 8 * (int64_t)sms;
    return launch_dependent(embed_runs_kernel<GT, VEC, ACC>, dim3((unsigned)grid), dim3(kThreads), 0,
                            s, a, side, chunk, segs);
}

template <int YT, int GT> cudaError_t grad_pick(const EmbedGradArgs &a, int sms, cudaStream_t s)
{
    const bool vec = rows_aligned(a.dy, a.dy_stride, YT, a.dim) &&
                     rows_aligned(a.grad, a.grad_stride, GT, a.dim);
    if (a.accumulate)
        return vec ? grad_go<YT, GT, true, true>(a, sms, s) : grad_go<YT, GT, false, true>(a, sms, s);
    return vec ? grad_go<YT, GT, true, false>(a, sms, s) : grad_go<YT, GT, false, false>(a, sms, s);
}

template <int YT>
cudaError_t grad_type(int32_t gdt, const EmbedGradArgs &a, int sms, cudaStream_t s)
{
    return gdt == F32 ? grad_pick<YT, F32>(a, sms, s)
                      : gdt == BF16 ? grad_pick<YT, BF16>(a, sms, s)
                                    : grad_pick<YT, F16>(a, sms, s);
}

}  // namespace

cudaError_t launch_embed(int32_t dt, const EmbedArgs &a, cudaStream_t s)
{
    if (a.tok.n <= 0 || a.dim <= 0) return cudaSuccess;
    return dt == F32 ? embed_pick<F32>(a, s) : dt == BF16 ? embed_pick<BF16>(a, s)
                                                          : embed_pick<F16>(a, s);
}

int64_t embed_grad_layout(EmbedGradArgs &a, char *base)
{
    // few tokens need no lists; the arrays then have no elements
    const int64_t n = a.tok.n <= kFewTokens ? 0 : a.tok.n;
    int64_t off = 0;
    auto take = [&](int64_t bytes) {
        char *p = base + off;
        off += (bytes + 255) / 256 * 256;
        return p;
    };
    const int64_t chunks = (n + sum_chunk(n) - 1) / sum_chunk(n);
    const int64_t segs = (a.dim + kCols - 1) / kCols;
    a.n_runs = reinterpret_cast<uint32_t *>(take(4));
    a.runs = reinterpret_cast<uint32_t *>(take(4 * chunks));
    const bool big = n > 0 && !sort_small(a);
    for (int i = 0; i < 2; ++i) {
        const int64_t len = i == 0 || big ? n : 0;
        a.key[i] = reinterpret_cast<uint32_t *>(take(4 * len));
        a.idx[i] = reinterpret_cast<uint32_t *>(take(4 * len));
    }
    a.hist = reinterpret_cast<uint32_t *>(take(big ? 4ll * 4 * 256 * kMaxSortBlocks : 0));
    a.part = reinterpret_cast<float *>(take(chunks * 2 * segs * kCols * 4));
    return off > 0 ? off : 256;
}

cudaError_t launch_embed_grad(int32_t ydt, int32_t gdt, const EmbedGradArgs &a, int sms,
                              cudaStream_t s)
{
    if (a.dim <= 0 || a.tok.rows <= 0) return cudaSuccess;
    if (a.tok.n <= 0 && a.accumulate) return cudaSuccess;
    return ydt == F32 ? grad_type<F32>(gdt, a, sms, s)
                      : ydt == BF16 ? grad_type<BF16>(gdt, a, sms, s)
                                    : grad_type<F16>(gdt, a, sms, s);
}

}  // namespace zgb

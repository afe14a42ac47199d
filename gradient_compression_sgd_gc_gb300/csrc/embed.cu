// embed.cu -- embedding lookup with scaling, and its gradient by sorted tokens.
//
//   lookup    out[t][:] = scale * table[id_t][:]
//   gradient  G[v][:]   = scale * sum_{t: id_t = v} dout[t][:]
//
// Both move bytes and compute next to nothing; the lookup reads the distinct
// rows and writes T rows, the gradient reads T rows and writes V.
#include <algorithm>

#include "lm_common.cuh"

namespace gc {
namespace {

// ---------------------------------------------------------------- columns

// A warp works on kCols columns of a row, 8 a lane.  Where every row starts on
// a boundary of 8 elements and D is a multiple of 8, lane l has the 8
// consecutive columns 8l..8l+7 (one 16- or 32-byte access); otherwise the
// columns l, l + 32, ... (element accesses, still contiguous over the warp).
constexpr int kCols = 256;

__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
    asm("ld.global.nc.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
        : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7])
        : "l"(p));
}
// Data that the thread will write.
__device__ __forceinline__ void load8_plain(const float* p, float (&f)[8]) {
    asm volatile("ld.global.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7])
                 : "l"(p)
                 : "memory");
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
    asm volatile("st.global.cs.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(f[0]), "f"(f[1]), "f"(f[2]),
                 "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
                 : "memory");
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&f)[8]) {
    Elem<__nv_bfloat16>::unpack(__ldg(reinterpret_cast<const uint4*>(p)), f);
}
__device__ __forceinline__ void load8_plain(const __nv_bfloat16* p, float (&f)[8]) {
    Elem<__nv_bfloat16>::unpack(__ldcg(reinterpret_cast<const uint4*>(p)), f);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&f)[8]) {
    __stcs(reinterpret_cast<uint4*>(p), Elem<__nv_bfloat16>::pack(f));
}

// The lane's columns of a row from c0 on; those beyond D keep their values.
template <typename T, bool VEC>
__device__ __forceinline__ void load_cols(const T* row, int64_t c0, int64_t D, int lane, float (&f)[8]) {
    if (VEC) {
        if (c0 + 8 * lane < D) load8(row + c0 + 8 * lane, f);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c0 + 32 * j + lane < D) f[j] = Elem<T>::load(row + c0 + 32 * j + lane);
    }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store_cols(T* row, int64_t c0, int64_t D, int lane, const float (&f)[8]) {
    if (VEC) {
        if (c0 + 8 * lane < D) store8(row + c0 + 8 * lane, f);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c0 + 32 * j + lane < D) row[c0 + 32 * j + lane] = Elem<T>::round_to(f[j]);
    }
}

// ---------------------------------------------------------------- lookup


struct LookupArgs {
    const void* table;
    const void* ids;
    void* out;
    int64_t ld_table, ld_out, T, V, D;
    int parts_log2;                // warps of a CTA that share one token, as a power of two
    float scale;
    int id64;
    int* status;
};

// One warp per (token, CHUNKS * kCols columns), its loads in flight together; a
// CTA's warps take the parts of one row, or of several where the rows are short.
// Two chunks, or one for rows that fit one (32768 tokens of 4096 bf16: 85, 64,
// 63, 69 us with 1, 2, 4, 8; 41 k of 320 fp32 into bf16 14.6, 11.3, 13.4, 21.6;
// 65536 of 128 bf16 11.6, 13.5, 18.3, 31.9).
template <typename TI, typename TO, bool VEC, int CHUNKS>
__global__ void __launch_bounds__(kThreads) k_embed_lookup(LookupArgs a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int parts = 1 << a.parts_log2;
    const int64_t t = (static_cast<int64_t>(blockIdx.x) * kWarpsPerBlock + warp) >> a.parts_log2;
    const int64_t c0 = (static_cast<int64_t>(blockIdx.y) * parts + (warp & (parts - 1))) * (CHUNKS * kCols);
    if (t >= a.T || c0 >= a.D) return;
    const int64_t id = load_id(a.ids, a.id64, t, a.V, a.status);
    float f[CHUNKS][8] = {};
    if (id >= 0) {
        const TI* row = static_cast<const TI*>(a.table) + id * a.ld_table;
#pragma unroll
        for (int k = 0; k < CHUNKS; ++k) load_cols<TI, VEC>(row, c0 + k * kCols, a.D, lane, f[k]);
#pragma unroll
        for (int k = 0; k < CHUNKS; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) f[k][j] *= a.scale;
    }
    TO* out = static_cast<TO*>(a.out) + t * a.ld_out;
#pragma unroll
    for (int k = 0; k < CHUNKS; ++k) store_cols<TO, VEC>(out, c0 + k * kCols, a.D, lane, f[k]);
}

// ---------------------------------------------------------------- gradient: order

// The tokens sorted by id, stable, without any exchange between CTAs of a
// launch.  Ids fall into classes, id mod B with B a power of two, so that the
// frequent low ids of a vocabulary spread over the classes; a CTA per class
// places its tokens.  It needs them in rising order, and the number of tokens
// of lower classes, which is where its own start:
//   few tokens: it reads all ids (they stay in L2) and picks its own;
//   many:       a first launch, a CTA per tile of kTile tokens, sorts each tile
//               by class and writes the tokens (place in the tile, number of
//               the id in its class) with the classes' starts.
// Reading everything costs B times the ids, the second launch 2 to 5 us.  Where
// the two cross depends on the table, since the zeroing of its last rows hides
// more of the longer sort: the whole gradient, cold L2, one launch against two,
//   tokens              2000        4000        6000        8000       10000
//   2500 x 1024      21.2  24.2  23.3  28.3  25.3  28.3  29.3  30.4  33.4  34.5
//   32003 x 1001     35.5  38.5  43.7  45.7  45.7  46.7  49.8  48.8  51.9  50.8
//   50000 x 768 bf16 25.2  30.3  28.4  31.4  31.4  32.4  33.4  32.4  35.5  34.4
//   131072 x 256     33.4  36.5  35.6  36.5  39.6  38.5  41.6  38.5  41.7  38.5
//   131072 x 2048     177   176   181   178   184   182   189   184   194   186
// The rule goes by the tokens alone, in the middle of the crossings: at its
// bound it gives up 2 us of 184 into the largest, 3 us of 28 into the smallest.
// Both launches place tokens the same way: a warp's tokens follow one another,
// per (warp, key) counts summed over warps and keys give each warp its first
// place for each key, and within 32 tokens a match gives the rank.
constexpr int64_t kFewTokens = 6 * 1024;
constexpr int kTile = 512;                  // tokens
constexpr int kTileThreads = 256;
constexpr int kTileWarps = kTileThreads / 32;
constexpr int kPerLane = kTile / kTileThreads;
constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kRangeBits = 11;
constexpr int kMaxRange = 1 << kRangeBits;  // ids per class: 16 x 2048 counts of 4 bytes of shared memory
constexpr int kMinClasses = 128;
constexpr int64_t kMaxTableRows = 1LL << 21;        // at most 1024 classes: 8 x 1024 counts in a tile's CTA

// Row order of the gradient's work: class by class, rising within a class.
struct Classes {
    int bits;                               // log2 B
    int64_t each, extra;                    // ids per class, classes with one more

    __host__ __device__ int64_t first(int64_t c) const { return c * each + (c < extra ? c : extra); }
};

struct GradArgs {
    const void* dout;
    const void* ids;
    void* dtable;
    int64_t ld_dout, ld_dtable, T, V, D;
    int64_t chunks, seg, nseg;     // columns / kCols; path items a segment; segments
    int tok_cost;                  // path items of one token; a row is one
    float scale;
    int id64, accumulate;
    Classes classes;
    int* status;
    // workspace; rows are counted in the classes' order
    int* row_start;                // [V + 1] first place of each row's tokens in `order`
    int* order;                    // [T] tokens sorted by row
    uint32_t* entries;             // [tiles][kTile] a tile's tokens sorted by class: place in the tile, number in the class
    int* starts;                   // [B + 1][tiles] where each class begins in a tile
    int64_t tiles;
    int2* split;                   // [nseg + 1] (row, place) where each segment begins
    unsigned* arrived;             // [3][nseg * chunks] parts of a shared row that are there
    float* carry;                  // [nseg][2][chunks * kCols] partial rows
    // rows from `zero_from` on are zeroed while the tokens are sorted, in pieces
    int64_t zero_from, pieces;
    int64_t piece_bytes, piece_pitch, zero_bytes;   // of a piece, to the next one, to the last one's end
    int elem;                      // bytes of an element of the table
};

// Lets the next kernel of this call start, and waits for the one before: its
// writes are there.
__device__ __forceinline__ void allow_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The place of this lane's key among the warp's tokens so far: counts[key] is
// the next one.  Lanes with the same key take consecutive places.
__device__ __forceinline__ int next_place(int* counts, uint32_t key, bool have, int lane) {
    const unsigned same = __match_any_sync(0xffffffffu, have ? key : 0xffffffffu);
    const int rank = __popc(same & ((1u << lane) - 1u));
    int at = 0;
    if (have) at = counts[key] + rank;
    __syncwarp();
    if (have && rank == 0) counts[key] += __popc(same);
    __syncwarp();
    return at;
}

template <typename I>
__global__ void __launch_bounds__(kTileThreads) k_embed_tiles(GradArgs a) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    __shared__ int warp_sum[kTileWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int B = 1 << a.classes.bits;
    int* counts = reinterpret_cast<int*>(smem_raw);         // [warps][B]
    int* mine = counts + warp * B;
    const int64_t tile = blockIdx.x, t0 = tile * kTile;
    const I* ids = static_cast<const I*>(a.ids);

    allow_next();
    uint32_t id[kPerLane];                  // all ones: absent
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
        const int64_t t = t0 + warp * (32 * kPerLane) + 32 * j + lane;
        const int64_t x = t < a.T ? static_cast<int64_t>(__ldg(ids + t)) : -1;
        if (x >= a.V && a.status) atomicExch(a.status, GC_ERR_INVALID);
        id[j] = static_cast<uint64_t>(x) < static_cast<uint64_t>(a.V) ? static_cast<uint32_t>(x) : 0xffffffffu;
    }
    for (int64_t k = tile * kTileThreads + tid; k < 3 * a.nseg * a.chunks; k += static_cast<int64_t>(gridDim.x) * kTileThreads)
        a.arrived[k] = 0;
    for (int c = tid; c < kTileWarps * B; c += kTileThreads) counts[c] = 0;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPerLane; ++j)
        if (id[j] != 0xffffffffu) atomicAdd(&mine[id[j] & (B - 1)], 1);
    __syncthreads();
    int start = 0;
    for (int c0 = 0; c0 < B; c0 += kTileThreads) {
        const int c = c0 + tid;
        int total = 0;
        if (c < B)
            for (int w = 0; w < kTileWarps; ++w) total += counts[w * B + c];
        int incl = total;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        __syncthreads();
        if (lane == 31) warp_sum[warp] = incl;
        __syncthreads();
        int before = 0, round = 0;
        for (int w = 0; w < kTileWarps; ++w) {
            if (w < warp) before += warp_sum[w];
            round += warp_sum[w];
        }
        if (c < B) {
            int at = start + before + incl - total;
            a.starts[c * a.tiles + tile] = at;
            for (int w = 0; w < kTileWarps; ++w) {
                const int n = counts[w * B + c];
                counts[w * B + c] = at;
                at += n;
            }
        }
        start += round;
    }
    if (tid == 0) a.starts[B * a.tiles + tile] = start;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
        const bool have = id[j] != 0xffffffffu;
        const int at = next_place(mine, id[j] & (B - 1), have, lane);
        if (have)
            a.entries[t0 + at] = static_cast<uint32_t>(warp * (32 * kPerLane) + 32 * j + lane) << kRangeBits |
                                 id[j] >> a.classes.bits;
    }
}

// Sorting leaves the memory idle, and most rows of a large table have no token.
// CTAs beside the sorting ones zero the table's last rows meanwhile, and the
// sums then write only those of them that have tokens (after this grid, so the
// order is certain).  The frequent ids of a vocabulary are low, so the last rows
// are the emptiest.  It pays while the writes take no longer than the sort,
// kZeroFew or kZeroMany bytes (one launch or two), and not where tokens fill
// the table, so only for T <= V, and a third of it at most.  Cold L2, without
// and with: 500 tokens into 131072 x 256 fp32 34.8 and 32.8 us, 24000 48.1 and
// 44.0, 65536 into 131072 x 2048 236.6 and 229.4 (248 with 96 MB, 252 with
// 128), 65536 into 5000 x 4096 133 and 143 if it were done there.  Two CTAs per
// SM: 64 MB in 152 CTAs takes 5 us longer, in 456 the same.
//
// A CTA's copies come from one piece of zeroed shared memory; the bytes before
// the first 16-byte boundary of a piece and after its last are stored singly.
constexpr int64_t kZeroFew = 32 << 20;
constexpr int64_t kZeroMany = 64 << 20;
constexpr int64_t kZeroPart = 3;
constexpr int kZeroCtas = 2 * 152;
constexpr int64_t kPieceBytes = 16384;      // of a table without gaps; else a row is a piece

__device__ __forceinline__ void zero_pieces(const GradArgs& a, int64_t part, int64_t parts, unsigned char* zeros) {
    for (int k = threadIdx.x; k < static_cast<int>(kPieceBytes / 16); k += kSortThreads)
        reinterpret_cast<uint4*>(zeros)[k] = make_uint4(0, 0, 0, 0);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
    if (threadIdx.x >= 32) return;
    const int lane = threadIdx.x;
    const uint32_t src = static_cast<uint32_t>(__cvta_generic_to_shared(zeros));
    char* const base = static_cast<char*>(a.dtable) + a.zero_from * a.ld_dtable * a.elem;
    for (int64_t k = part; k < a.pieces; k += parts) {
        char* p = base + k * a.piece_pitch;
        const int n = static_cast<int>(min(a.piece_bytes, a.zero_bytes - k * a.piece_pitch));
        const int head = min(n, static_cast<int>(-reinterpret_cast<uintptr_t>(p) & 15));
        const int body = (n - head) & ~15, tail = n - head - body;
        if (2 * lane < head) *reinterpret_cast<uint16_t*>(p + 2 * lane) = 0;
        if (2 * lane < tail) *reinterpret_cast<uint16_t*>(p + head + body + 2 * lane) = 0;
        if (lane == 0)
            for (int at = 0; at < body; at += static_cast<int>(kPieceBytes))
                asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                                 __cvta_generic_to_global(p + head + at)),
                             "r"(src), "r"(min(body - at, static_cast<int>(kPieceBytes)))
                             : "memory");
    }
    if (lane == 0) {
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
}

// Calls f(have, number in the class, token) for the tokens of class c in tiles
// [tile0, tile1), in their order, 32 at a time.  The bounds of 32 tiles are
// read at once; a lane finds the tile of its token by bisection over the sums
// of the tiles' counts.
template <typename F>
__device__ __forceinline__ void for_tiled(const GradArgs& a, int64_t c, int64_t tile0, int64_t tile1, int lane, F f) {
    for (int64_t t0 = tile0; t0 < tile1; t0 += 32) {
        int from = 0, count = 0;
        if (t0 + lane < tile1) {
            from = a.starts[c * a.tiles + t0 + lane];
            count = a.starts[(c + 1) * a.tiles + t0 + lane] - from;
        }
        int incl = count;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        const int total = __shfl_sync(0xffffffffu, incl, 31), first = from - (incl - count);
        for (int k = 0; k < total; k += 32) {
            const int i = k + lane;
            int tile = 0;                   // the number of tiles whose sums are at most i
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1)
                if (__shfl_sync(0xffffffffu, incl, tile + o - 1) <= i) tile += o;
            const int place = __shfl_sync(0xffffffffu, first, tile & 31) + i;
            const bool have = i < total;
            const int64_t t = (t0 + tile) * kTile;
            const uint32_t e = have ? a.entries[t + place] : 0;
            f(have, e & (kMaxRange - 1), static_cast<int>(t + (e >> kRangeBits)));
        }
    }
}

// The same from the ids [t0, t1) themselves; lower(valid) is called for every
// token with whether its class is below c.
template <typename I, typename F, typename L>
__device__ __forceinline__ void for_scanned(const GradArgs& a, uint32_t c, int64_t t0, int64_t t1, int lane, F f, L lower) {
    constexpr int kLoads = 4;
    const uint32_t mask = (1u << a.classes.bits) - 1u;
    for (int64_t t = t0; t < t1; t += 32 * kLoads) {
        int64_t id[kLoads];
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int64_t i = t + 32 * j + lane;
            id[j] = i < t1 ? static_cast<int64_t>(__ldg(static_cast<const I*>(a.ids) + i)) : -1;
        }
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const bool valid = static_cast<uint64_t>(id[j]) < static_cast<uint64_t>(a.V);
            const uint32_t cls = static_cast<uint32_t>(id[j]) & mask;
            lower(valid && cls < c, id[j]);
            const bool have = valid && cls == c;
            if (__any_sync(0xffffffffu, have))
                f(have, static_cast<uint32_t>(id[j]) >> a.classes.bits, static_cast<int>(t + 32 * j + lane));
        }
    }
}

__device__ __forceinline__ int64_t path_of(const GradArgs& a, int64_t row, int64_t place) {
    return a.tok_cost * place + row;
}

template <typename I, bool TILED>
__global__ void __launch_bounds__(kSortThreads) k_embed_order(GradArgs a) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    __shared__ int warp_sum[kSortWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int B = 1 << a.classes.bits;
    if (blockIdx.x >= B) {
        allow_next();
        zero_pieces(a, blockIdx.x - B, gridDim.x - B, smem_raw);
        return;
    }
    const int64_t lo = a.classes.first(blockIdx.x);          // the class's first row
    const int n_ids = static_cast<int>(a.classes.first(blockIdx.x + 1) - lo);
    int* const all = reinterpret_cast<int*>(smem_raw);      // [warps][n_ids] counts
    int* const first_of = all + kSortWarps * n_ids;         // [n_ids + 1] where each id's tokens begin; then the class's end
    int* const counts = all + warp * n_ids;

    allow_next();
    for (int k = tid; k < kSortWarps * n_ids; k += kSortThreads) all[k] = 0;
    // a warp's tokens: a run of tiles, or of ids
    const int64_t units = TILED ? a.tiles : (a.T + 31) / 32, per = (units + kSortWarps - 1) / kSortWarps;
    const int64_t unit0 = min(units, warp * per), unit1 = min(units, unit0 + per);
    auto for_tokens = [&](auto f, auto lower) {
        if constexpr (TILED) for_tiled(a, blockIdx.x, unit0, unit1, lane, f);
        else for_scanned<I>(a, blockIdx.x, unit0 * 32, min(a.T, unit1 * 32), lane, f, lower);
    };
    int below = 0;
    if (TILED) {
        wait_previous();
        for (int64_t t = tid; t < a.tiles; t += kSortThreads) below += a.starts[blockIdx.x * a.tiles + t];
    } else {
        for (int64_t k = static_cast<int64_t>(blockIdx.x) * kSortThreads + tid; k < 3 * a.nseg * a.chunks;
             k += static_cast<int64_t>(B) * kSortThreads)
            a.arrived[k] = 0;
    }
    __syncthreads();
    for_tokens(
        [&](bool have, uint32_t key, int) {
            if (have) atomicAdd(&counts[key], 1);
        },
        [&](bool is_lower, int64_t id) {
            below += is_lower;
            if (id >= a.V && blockIdx.x == 0 && a.status) atomicExch(a.status, GC_ERR_INVALID);
        });
    below = __reduce_add_sync(0xffffffffu, below);
    if (lane == 0) warp_sum[warp] = below;
    __syncthreads();
    int start = 0;
    for (int w = 0; w < kSortWarps; ++w) start += warp_sum[w];

    // kSortThreads ids a round: their counts, the exclusive prefix, then each
    // warp's first place for each
    for (int l0 = 0; l0 < n_ids; l0 += kSortThreads) {
        const int l = l0 + tid;
        int total = 0;
        if (l < n_ids)
            for (int w = 0; w < kSortWarps; ++w) total += all[w * n_ids + l];
        int incl = total;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        __syncthreads();
        if (lane == 31) warp_sum[warp] = incl;
        __syncthreads();
        int before = 0, round = 0;
        for (int w = 0; w < kSortWarps; ++w) {
            if (w < warp) before += warp_sum[w];
            round += warp_sum[w];
        }
        const int first = start + before + incl - total;
        if (l < n_ids) {
            int at = first;
            for (int w = 0; w < kSortWarps; ++w) {
                const int c = all[w * n_ids + l];
                all[w * n_ids + l] = at;
                at += c;
            }
            a.row_start[lo + l] = first;
            first_of[l] = first;
        }
        start += round;
    }
    if (tid == 0) {
        first_of[n_ids] = start;
        if (lo + n_ids == a.V) a.row_start[a.V] = start;
    }
    __syncthreads();
    // the segments that begin within this class's path
    const int64_t p0 = path_of(a, lo, first_of[0]), p1 = path_of(a, lo + n_ids, first_of[n_ids]);
    for (int64_t m = (p0 + a.seg - 1) / a.seg + tid; m * a.seg < p1; m += kSortThreads) {
        int l = 0, r = n_ids;               // path_of(l) <= m * seg < path_of(r)
        while (r - l > 1) {
            const int mid = (l + r) >> 1;
            if (path_of(a, lo + mid, first_of[mid]) <= m * a.seg) l = mid;
            else r = mid;
        }
        const int64_t into = (m * a.seg - path_of(a, lo + l, first_of[l])) >> (a.tok_cost - 1);
        a.split[m] = make_int2(static_cast<int>(lo + l),
                               static_cast<int>(min(static_cast<int64_t>(first_of[l + 1]), first_of[l] + into)));
    }
    if (lo + n_ids == a.V)
        for (int64_t m = (p1 + a.seg - 1) / a.seg + tid; m <= a.nseg; m += kSortThreads)
            a.split[m] = make_int2(static_cast<int>(a.V), first_of[n_ids]);
    for_tokens(
        [&](bool have, uint32_t key, int token) {
            const int at = next_place(counts, key, have, lane);
            if (have) a.order[at] = token;
        },
        [](bool, int64_t) {});
}

// ---------------------------------------------------------------- gradient: sums

// The work is a path over rows and tokens: a row's tokens, then the row's
// write.  It is cut into nseg segments of equal length, whatever the tokens'
// frequencies; a warp takes one segment for kCols columns.  A row that lies in
// one segment is written there.  A row that spans several has its partial sums
// (fp32) left in the workspace, and the warp that finds all the others' parts
// there adds them in segment order and writes the row, so the result does not
// depend on which warp is last.
template <typename TO, bool VEC>
__device__ __forceinline__ void write_row(const GradArgs& a, TO* out, int64_t c0, int lane, float (&acc)[8], bool any) {
    if (a.accumulate && !any) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] *= a.scale;
    if (a.accumulate) {
        float old[8] = {};
        if (VEC) {
            if (c0 + 8 * lane < a.D) load8_plain(out + c0 + 8 * lane, old);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c0 + 32 * j + lane < a.D) old[j] = Elem<TO>::load_plain(out + c0 + 32 * j + lane);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] += old[j];
    }
    store_cols<TO, VEC>(out, c0, a.D, lane, acc);
}

__device__ __forceinline__ float* carry_of(const GradArgs& a, int64_t m, int slot, int64_t c0, int lane) {
    return a.carry + ((m * 2 + slot) * a.chunks * kCols + c0) + 8 * lane;
}

// One part of several has been written; whether all `count` of them are there.
__device__ __forceinline__ bool last_to_arrive(unsigned* counter, int64_t count, int lane) {
    __threadfence();
    __syncwarp();
    unsigned seen = 0;
    if (lane == 0) seen = atomicAdd(counter, 1u);
    seen = __shfl_sync(0xffffffffu, seen, 0);
    if (seen + 1 != static_cast<unsigned>(count)) return false;
    __threadfence();
    return true;
}

// This segment's part of a row that segments first..last share.  The parts are
// joined in groups of kJoin segments, then the groups, each sum in its order by
// the warp that finds its terms complete: a token that fills a tenth of a batch
// has hundreds of parts.
constexpr int kJoin = 32;

template <typename TO, bool VEC>
__device__ __forceinline__ void shared_row(const GradArgs& a, TO* out, int64_t m, int64_t first, int64_t last, int64_t chunk,
                                           int lane, float4 lo, float4 hi, bool any) {
    const int64_t c0 = chunk * kCols, counters = a.nseg * a.chunks;
    auto place = [&](int64_t k) { return reinterpret_cast<float4*>(carry_of(a, k, k == first ? 1 : 0, c0, lane)); };
    auto put = [&](int64_t k, float4 x, float4 y) {
        __stcg(place(k), x);
        __stcg(place(k) + 1, y);
    };
    float sum[8];
    auto add_up = [&](int64_t from, int64_t to, int64_t step) {
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
#pragma unroll 8
        for (int64_t k = from; k <= to; k += step) {
            const float4 x = load_ordered(place(k)), y = load_ordered(place(k) + 1);
            sum[0] += x.x, sum[1] += x.y, sum[2] += x.z, sum[3] += x.w;
            sum[4] += y.x, sum[5] += y.y, sum[6] += y.z, sum[7] += y.w;
        }
    };
    const int64_t group = (m - first) / kJoin, head = first + group * kJoin, tail = min(last, head + kJoin - 1);
    put(m, lo, hi);
    // a segment may be the first of this row's parts and the head of another's group
    unsigned* counter = a.arrived + (group == 0 ? 0 : counters) + head * a.chunks + chunk;
    if (!last_to_arrive(counter, tail - head + 1, lane)) return;
    add_up(head, tail, 1);
    const int64_t groups = (last - first) / kJoin + 1;
    if (groups > 1) {
        put(head, make_float4(sum[0], sum[1], sum[2], sum[3]), make_float4(sum[4], sum[5], sum[6], sum[7]));
        if (!last_to_arrive(a.arrived + 2 * counters + first * a.chunks + chunk, groups, lane)) return;
        add_up(first, last, kJoin);
    }
    write_row<TO, VEC>(a, out, c0, lane, sum, any);
}

constexpr int kGroup = 4;           // token rows of one asynchronous copy group
constexpr int kRing = 2 * kGroup;   // places of a warp: one group is added while the other arrives
constexpr int kPlace = kCols + 16;  // elements of a place
constexpr int kSumCtas = 3;         // resident per SM

// Starts the copy of n columns of a token row to a place of a warp's ring, in
// 16-byte vectors, and returns where in the place they begin.  Rows that start
// anywhere are copied from the aligned address below (`before` elements of the
// buffer lie there at least), the last vector only as far as the columns go.
template <typename T, bool VEC>
__device__ __forceinline__ int copy_cols(const T* from, int n, int64_t before, int lane, T* place) {
    constexpr int kPer = 16 / sizeof(T), kVecs = kCols / kPer;
    const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(place)) + 16 * lane;
    if (VEC) {
        const T* src = from + kPer * lane;
#pragma unroll
        for (int j = 0; j < kVecs / 32; ++j)
            if (n == kCols || (32 * j + lane) * kPer < n)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + 512 * j),
                             "l"(__cvta_generic_to_global(src + 32 * kPer * j))
                             : "memory");
        return 0;
    }
    const int shift = row_shift(from);
    if (before < shift) {                   // the buffer's first elements
        for (int c = lane; c < n; c += 32) place[shift + c] = from[c];
        return shift;
    }
    const T* src = from - shift + kPer * lane;
    int left = (n + shift - kPer * lane) * static_cast<int>(sizeof(T));  // bytes from this lane's vector on
#pragma unroll
    for (int j = 0; j < kVecs / 32 + 1; ++j, left -= 512)
        if (left > 0 && (j < kVecs / 32 || lane == 0))
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + 512 * j),
                         "l"(__cvta_generic_to_global(src + 32 * kPer * j)), "r"(min(left, 16))
                         : "memory");
    return shift;
}

// Adds the lane's columns from a place of the ring; those beyond the last add
// what the place happened to hold to sums that are not written.
template <typename T, bool VEC>
__device__ __forceinline__ void add_cols(const T* place, int lane, float (&acc)[8]) {
    if (VEC) {
        float f[8];
        const uint4* p = reinterpret_cast<const uint4*>(place + 8 * lane);
        if (sizeof(T) == 2) {
            Elem<__nv_bfloat16>::unpack(p[0], f);
        } else {
            float g[4];
            Elem<float>::unpack(p[0], g);
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = g[j];
            Elem<float>::unpack(p[1], g);
#pragma unroll
            for (int j = 0; j < 4; ++j) f[4 + j] = g[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] += f[j];
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] += static_cast<float>(place[32 * j + lane]);
    }
}

template <typename TI, typename TO, bool VEC>
__global__ void __launch_bounds__(kThreads, kSumCtas) k_embed_sum(GradArgs a) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    TI* ring = reinterpret_cast<TI*>(smem_raw) + warp * kRing * kPlace;
    const unsigned w = blockIdx.x * kWarpsPerBlock + warp, chunks = static_cast<unsigned>(a.chunks);
    const int64_t m = w / chunks, chunk = w % chunks;
    if (m >= a.nseg) return;
    wait_previous();
    const int2 from = a.split[m], to = a.split[m + 1];
    const int64_t c0 = chunk * kCols;
    int64_t row = from.x;
    int place = from.y;
    if (row == a.V) return;                // past the path's end (absent tokens)

    // the row's id and where it is written
    const int64_t B = 1LL << a.classes.bits;
    const int64_t big = a.classes.extra * (a.classes.each + 1);
    int64_t cls = row < big ? row / (a.classes.each + 1) : a.classes.extra + (row - big) / max(a.classes.each, int64_t(1));
    int64_t id = ((row - a.classes.first(cls)) << a.classes.bits) + cls;
    TO* out = static_cast<TO*>(a.dtable) + id * a.ld_dtable;

    // row_start[base + 1 + lane]: the ends of 32 rows
    int64_t base = row;
    int ends = a.row_start[min(a.V, base + 1 + lane)];
    int row_first = a.row_start[row];      // where the current row's tokens begin
    int end = __shfl_sync(0xffffffffu, ends, 0);
    bool began = path_of(a, row, row_first) >= m * a.seg;   // the row, in this segment
    auto advance = [&]() {
        ++row;
        id += B;
        out += B * a.ld_dtable;
        if (id >= a.V) {
            id = ++cls;
            out = static_cast<TO*>(a.dtable) + id * a.ld_dtable;
        }
        row_first = end;
        began = true;
        if (row - base == 32) {
            base = row;
            ends = a.row_start[min(a.V, base + 1 + lane)];
        }
        end = __shfl_sync(0xffffffffu, ends, static_cast<int>(row - base));
    };
    float acc[8] = {};
    // writes rows from the current one on that have no token left, up to `last`
    auto finish = [&](int64_t last) {
        if (end > row_first || !began) {
            if (began) {
                write_row<TO, VEC>(a, out, c0, lane, acc, true);
            } else {
                shared_row<TO, VEC>(a, out, m, path_of(a, row, row_first) / a.seg, m, chunk, lane,
                                    make_float4(acc[0], acc[1], acc[2], acc[3]),
                                    make_float4(acc[4], acc[5], acc[6], acc[7]), end > row_first);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
            advance();
        }
        const float none[8] = {};
        while (row < last && end == place) {
            if (!a.accumulate && id < a.zero_from) store_cols<TO, VEC>(out, c0, a.D, lane, none);
            advance();
        }
    };

    // groups of tokens, one copied while the one before is added; `tok` holds 32
    // tokens of the order, the next 32 are read meanwhile
    const int n = static_cast<int>(min(static_cast<int64_t>(kCols), a.D - c0));
    const TI* dout = static_cast<const TI*>(a.dout) + c0;
    int ahead = place, tok = 0, tok_next = 0;
    if (lane < to.y - place) tok = a.order[place + lane];
    if (lane < to.y - place - 32) tok_next = a.order[place + 32 + lane];
    uint64_t shifts = 0;                    // 4 bits for each place of the ring
    auto copy_group = [&]() {
#pragma unroll
        for (int k = 0; k < kGroup; ++k) {
            if (ahead + k < to.y) {
                const int i = ahead + k - from.y, slot = i % kRing;
                const int64_t at = static_cast<int64_t>(__shfl_sync(0xffffffffu, tok, i % 32)) * static_cast<int>(a.ld_dout);
                const int shift = copy_cols<TI, VEC>(dout + at, n, at + c0, lane, ring + slot * kPlace);
                if (!VEC) shifts = (shifts & ~(15ull << (4 * slot))) | static_cast<uint64_t>(shift) << (4 * slot);
            }
        }
        ahead += kGroup;
        if ((ahead - from.y) % 32 == 0) {
            tok = tok_next;
            if (lane < to.y - ahead - 32) tok_next = a.order[ahead + 32 + lane];
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    copy_group();
    while (place < to.y) {
        copy_group();
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncwarp();
        const int stop = min(to.y, place + kGroup);
        while (place < stop) {
            if (place == end) finish(a.V);
            const int run = min(end, stop);
            for (; place < run; ++place) {
                const int slot = (place - from.y) % kRing;
                add_cols<TI, VEC>(ring + slot * kPlace + (VEC ? 0 : static_cast<int>(shifts >> (4 * slot)) & 15), lane, acc);
            }
        }
        __syncwarp();
    }
    if (row < to.x && place == end) finish(to.x);
    // a row that a later segment ends, if its path has begun here
    if (row < a.V) {
        const int64_t p0 = path_of(a, row, row_first);
        if (p0 < (m + 1) * a.seg)
            shared_row<TO, VEC>(a, out, m, p0 / a.seg, (path_of(a, row + 1, end) - 1) / a.seg, chunk, lane,
                                make_float4(acc[0], acc[1], acc[2], acc[3]), make_float4(acc[4], acc[5], acc[6], acc[7]),
                                end > row_first);
    }
}

// ---------------------------------------------------------------- host

// Segments x column chunks of embed_grad.  Where the 24 warps that are resident
// on each of 152 SMs get segments of at most kLongSeg items, that many: a
// segment costs some 3 us to start (19465 tokens into 4507 x 1280: 30 us against
// 36 with four times as many).  Above, four times as many, which evens out hot
// and empty segments (65536 tokens into 131072 x 2048: 253 us against 266 with
// twice and 262 with eight times as many).  The workspace depends on it, so it
// goes by the sizes alone and not by the device.
constexpr int64_t kSumWarps = 152 * 96;
constexpr int64_t kResidentWarps = 152 * 24;
constexpr int64_t kLongSeg = 128;
constexpr int64_t kMinSeg = 16;   // above any cost, so that every segment moves on by a token or a row

struct GradPlan {
    int64_t chunks, seg, nseg;
    Classes classes;
    int64_t tiles;
    size_t row_start, order, entries, starts, split, arrived, carry, bytes;   // offsets, total
};

size_t up16(size_t n) { return (n + 15) & ~static_cast<size_t>(15); }

// Classes of V ids: kMinClasses unless their ranges are too long, none of them
// empty.
Classes make_classes(int64_t V) {
    Classes c;
    c.bits = 0;
    while ((2LL << c.bits) <= V && ((1 << c.bits) < kMinClasses || V > (static_cast<int64_t>(kMaxRange) << c.bits))) ++c.bits;
    c.each = V >> c.bits;
    c.extra = V & ((1LL << c.bits) - 1);
    return c;
}

// Costs: a token counts as a table row, as two where it has twice the bytes of
// one.  Half the bytes of one count as much: a segment of tokens alone waits for
// its copies (12000 bf16 tokens into 131072 x 256 fp32: 40.0 us against 43.5
// with a half, 39.2 with two; 65536 into 131072 x 2048: 230.6, 236.2, 236.2).
bool grad_plan(int64_t T, int64_t V, int64_t D, int tok_cost, GradPlan* p) {
    if (T < 0 || T > GC_MAX_TOKENS || V < 1 || V > kMaxTableRows || D < 0 || D > (1LL << 31)) return false;
    p->classes = make_classes(V);
    p->tiles = (T + kTile - 1) / kTile;
    if (p->tiles < 1) p->tiles = 1;
    p->chunks = (D + kCols - 1) / kCols;
    if (p->chunks < 1) p->chunks = 1;
    const int64_t path = T * tok_cost + V;
    auto cut = [&](int64_t warps) {
        const int64_t want = warps / p->chunks > 1 ? warps / p->chunks : 1;
        return (path + want - 1) / want;
    };
    p->seg = cut(kResidentWarps);
    if (p->seg > kLongSeg) p->seg = cut(kSumWarps);
    if (p->seg < kMinSeg) p->seg = kMinSeg;
    p->nseg = (path + p->seg - 1) / p->seg;
    size_t at = 0;
    p->row_start = at, at = up16(at + sizeof(int) * (V + 1));
    p->order = at, at = up16(at + sizeof(int) * T);
    p->entries = at, at = up16(at + sizeof(uint32_t) * p->tiles * kTile);
    p->starts = at, at = up16(at + sizeof(int) * ((1LL << p->classes.bits) + 1) * p->tiles);
    p->split = at, at = up16(at + sizeof(int2) * (p->nseg + 1));
    p->arrived = at, at = up16(at + sizeof(unsigned) * 3 * p->nseg * p->chunks);
    p->carry = at, at = up16(at + sizeof(float) * p->nseg * 2 * p->chunks * kCols);
    p->bytes = at;
    return true;
}

template <typename TI, typename TO, int CHUNKS>
int launch_lookup(LookupArgs a, bool vec, cudaStream_t s) {
    const int64_t parts = (a.D + CHUNKS * kCols - 1) / (CHUNKS * kCols);
    a.parts_log2 = 0;
    while (a.parts_log2 < 3 && (1 << a.parts_log2) < parts) ++a.parts_log2;
    const int64_t per_cta = kWarpsPerBlock >> a.parts_log2;
    const int64_t x = (a.T + per_cta - 1) / per_cta, y = (parts + (1 << a.parts_log2) - 1) >> a.parts_log2;
    if (x > 0x7fffffffLL || y > 65535) return GC_ERR_INVALID;
    const dim3 grid(static_cast<unsigned>(x), static_cast<unsigned>(y));
    if (vec)
        k_embed_lookup<TI, TO, true, CHUNKS><<<grid, kThreads, 0, s>>>(a);
    else
        k_embed_lookup<TI, TO, false, CHUNKS><<<grid, kThreads, 0, s>>>(a);
    return launch_status();
}

template <typename TI, typename TO>
int launch_lookup(const LookupArgs& a, bool vec, cudaStream_t s) {
    return a.D <= kCols ? launch_lookup<TI, TO, 1>(a, vec, s) : launch_lookup<TI, TO, 2>(a, vec, s);
}

// Launches a kernel that may start while the stream's previous one runs and
// waits for it itself.
int launch_next(void (*kernel)(GradArgs), unsigned blocks, int threads, size_t smem, const GradArgs& a, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) {
        cudaGetLastError();
        return GC_ERR_CUDA;
    }
    return GC_OK;
}

template <typename TI, typename TO>
int launch_sum(const GradArgs& a, bool vec, cudaStream_t s) {
    const unsigned blocks = static_cast<unsigned>((a.nseg * a.chunks + kWarpsPerBlock - 1) / kWarpsPerBlock);
    const int smem = kWarpsPerBlock * kRing * kPlace * static_cast<int>(sizeof(TI));
    auto kernel = vec ? k_embed_sum<TI, TO, true> : k_embed_sum<TI, TO, false>;
    if (allow_smem(kernel, smem, smem) != GC_OK) return GC_ERR_CUDA;
    return launch_next(kernel, blocks, kThreads, smem, a, s);
}

// Shared memory of a sorting CTA whose class has `ids` ids: counts of each warp,
// and where each id's tokens begin.
constexpr size_t order_bytes(int64_t ids) { return ((kSortWarps + 1) * ids + 1) * sizeof(int); }

// Whether every row of p starts on a boundary of 8 elements.
bool rows_aligned(const void* p, int64_t ld, int type) { return aligned_to(p, 8 * type_bytes(type)) && ld % 8 == 0; }

}  // namespace
}  // namespace gc

using namespace gc;

extern "C" {

int embed_lookup(const void* table, gc_dtype table_type, int64_t ld_table, const void* ids, gc_id_type id_type, void* out,
                 gc_dtype out_type, int64_t ld_out, int64_t T, int64_t V, int64_t D, float scale, int* d_status,
                 gc_stream_t stream) {
    if (T < 0 || D < 0 || V < 1 || V >= (1LL << 31) || ld_table < D || ld_out < D || !valid_type(table_type) ||
        !valid_type(out_type) || !valid_id_type(id_type) || !isfinite(scale))
        return GC_ERR_INVALID;
    if (T == 0 || D == 0) return GC_OK;
    if (!table || !ids || !out) return GC_ERR_INVALID;
    if (!aligned_to(table, type_bytes(table_type)) || !aligned_to(out, type_bytes(out_type)) ||
        !aligned_to(ids, id_type == GC_I64 ? 8 : 4) || !aligned_to(d_status, 4))
        return GC_ERR_ALIGN;
    LookupArgs a;
    a.table = table, a.ids = ids, a.out = out;
    a.ld_table = ld_table, a.ld_out = ld_out, a.T = T, a.V = V, a.D = D;
    a.scale = scale;
    a.id64 = id_type == GC_I64;
    a.status = d_status;
    const bool vec = D % 8 == 0 && rows_aligned(table, ld_table, table_type) && rows_aligned(out, ld_out, out_type);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (table_type == GC_F32)
        return out_type == GC_F32 ? launch_lookup<float, float>(a, vec, s) : launch_lookup<float, __nv_bfloat16>(a, vec, s);
    return out_type == GC_F32 ? launch_lookup<__nv_bfloat16, float>(a, vec, s)
                              : launch_lookup<__nv_bfloat16, __nv_bfloat16>(a, vec, s);
}

size_t embed_grad_workspace_bytes(int64_t T, int64_t V, int64_t D) {
    // the larger one over the costs of the element types
    size_t most = 0;
    GradPlan p;
    for (int tok = 1; tok <= 2; ++tok) {
        if (!grad_plan(T, V, D, tok, &p)) return 0;
        most = p.bytes > most ? p.bytes : most;
    }
    return most;
}

int embed_grad(const void* dout, gc_dtype dout_type, int64_t ld_dout, const void* ids, gc_id_type id_type, void* dtable,
               gc_dtype table_type, int64_t ld_dtable, int64_t T, int64_t V, int64_t D, float scale, int accumulate,
               void* workspace, size_t workspace_bytes, int* d_status, gc_stream_t stream) {
    if (D < 0 || ld_dout < D || ld_dout > 0x7fffffffLL || ld_dtable < D || !valid_type(dout_type) || !valid_type(table_type) ||
        !valid_id_type(id_type) || !isfinite(scale) || (accumulate != 0 && accumulate != 1))
        return GC_ERR_INVALID;
    GradPlan p;
    const int tok_cost = dout_type == GC_F32 && table_type == GC_BF16 ? 2 : 1;
    if (!grad_plan(T, V, D, tok_cost, &p)) return GC_ERR_INVALID;
    if (D == 0 || (T == 0 && accumulate)) return GC_OK;
    if (!dtable || !workspace || (T > 0 && (!dout || !ids)) || workspace_bytes < p.bytes) return GC_ERR_INVALID;
    if (!aligned_to(dout, type_bytes(dout_type)) || !aligned_to(dtable, type_bytes(table_type)) ||
        !aligned_to(ids, id_type == GC_I64 ? 8 : 4) || !aligned16(workspace) || !aligned_to(d_status, 4))
        return GC_ERR_ALIGN;
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    GradArgs a;
    a.dout = dout, a.ids = ids, a.dtable = dtable;
    a.ld_dout = ld_dout, a.ld_dtable = ld_dtable, a.T = T, a.V = V, a.D = D;
    a.chunks = p.chunks, a.seg = p.seg, a.nseg = p.nseg;
    a.tok_cost = tok_cost;
    a.scale = scale;
    a.id64 = id_type == GC_I64;
    a.accumulate = accumulate;
    a.status = d_status;
    a.row_start = reinterpret_cast<int*>(ws + p.row_start);
    a.order = reinterpret_cast<int*>(ws + p.order);
    a.entries = reinterpret_cast<uint32_t*>(ws + p.entries);
    a.starts = reinterpret_cast<int*>(ws + p.starts);
    a.classes = p.classes, a.tiles = p.tiles;
    a.split = reinterpret_cast<int2*>(ws + p.split);
    a.arrived = reinterpret_cast<unsigned*>(ws + p.arrived);
    a.carry = reinterpret_cast<float*>(ws + p.carry);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);

    const int B = 1 << a.classes.bits;
    const bool tiled = T > kFewTokens;
    a.elem = type_bytes(table_type);
    const int64_t row_bytes = D * a.elem;
    const int64_t zero_rows =
        accumulate || T > V ? 0 : std::min<int64_t>(V / kZeroPart, (tiled ? kZeroMany : kZeroFew) / row_bytes);
    a.zero_from = V - zero_rows;
    a.zero_bytes = zero_rows > 0 ? (zero_rows - 1) * ld_dtable * a.elem + row_bytes : 0;
    a.piece_bytes = ld_dtable == D ? kPieceBytes : row_bytes;
    a.piece_pitch = ld_dtable == D ? kPieceBytes : ld_dtable * a.elem;
    a.pieces = (a.zero_bytes + a.piece_pitch - 1) / a.piece_pitch;
    const int zero_ctas = static_cast<int>(std::min<int64_t>(kZeroCtas, a.pieces));
    const size_t smem = std::max<size_t>(kPieceBytes, order_bytes(a.classes.each + 1));
    auto order = tiled ? k_embed_order<int, true> : a.id64 ? k_embed_order<long long, false> : k_embed_order<int, false>;
    if (allow_smem(order, smem, order_bytes(kMaxRange + 1)) != GC_OK) return GC_ERR_CUDA;
    if (tiled) {
        auto tiles = a.id64 ? k_embed_tiles<long long> : k_embed_tiles<int>;
        tiles<<<static_cast<unsigned>(a.tiles), kTileThreads, kTileWarps * B * sizeof(int), s>>>(a);
        if (launch_status() != GC_OK || launch_next(order, B + zero_ctas, kSortThreads, smem, a, s) != GC_OK)
            return GC_ERR_CUDA;
    } else {
        order<<<B + zero_ctas, kSortThreads, smem, s>>>(a);
        if (launch_status() != GC_OK) return GC_ERR_CUDA;
    }

    const bool vec = D % 8 == 0 && (T == 0 || rows_aligned(dout, ld_dout, dout_type)) &&
                     rows_aligned(dtable, ld_dtable, table_type);
    if (dout_type == GC_F32)
        return table_type == GC_F32 ? launch_sum<float, float>(a, vec, s) : launch_sum<float, __nv_bfloat16>(a, vec, s);
    return table_type == GC_F32 ? launch_sum<__nv_bfloat16, float>(a, vec, s)
                                : launch_sum<__nv_bfloat16, __nv_bfloat16>(a, vec, s);
}

}  // extern "C"

// dense.cuh -- dense attention: the causal prompt pass and its backward, and the
// decode step over a shared prefix.  Work items, their enumeration and the
// launchers shared by the CUDA-core and the tensor-core kernels.
//
// Rows.  The G query heads of a group read the same keys, so a tile's rows are
// (token, head) pairs: row r is token r / G and head g*G + r % G.  q's layout
// [.., token, head, d] makes such a tile one box of consecutive memory per token.
#pragma once

#include <utility>

#include "hsa_internal.cuh"

namespace hsa {
namespace dense {

constexpr int32_t kKDense = 12;  // DevStatus::where of these kernels (KernelId goes to 11)
constexpr int kSimtRows = 64;    // rows and keys of a CUDA-core tile
constexpr int kNoMask = 0x3fffffff;  // causal offset of an item whose keys are all visible

// two FMAs in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}

// Geometry and tensors of one call (passed to the kernels by value).
struct Args {
    int decode;                  // 0: prompt pass, 1: decode over a shared prefix
    int B, L, hq, hkv, G;        // decode: L = P (prefix tokens)
    int tok;                     // tokens per row tile
    int off_by_one;
    float scale, scale_log2;     // 1 / sqrt(d), and that times log2(e)
    // prompt pass
    const int4 *plan;            // packed: {sequence's first token, its length, item's first token, split},
    const int32_t *plan_n;       //         dearest first (else null), and the entries in it
    int tiles;                   // not packed: items per batch row
    // decode
    int cap;                     // tokens of a sequence's own cache
    const int32_t *lens;         // [B]
    // The prefix is cut into pre_slots slots of pre_sub keys, each own cache into suf_slots of
    // suf_sub; an item takes one slot, whose attention is one partial.
    int pre_tiles, pre_sub, pre_slots;
    int suf_sub, suf_slots;
    int split;                   // tensor cores, decode or not packed: an item's two streams have the same rows
                                 // and split the keys (else they have a tile of rows each)
    // tensors: 0 = the prompt's (or the prefix's) keys and values, 1 = the own caches'
    const void *q, *k[2], *v[2];
    int64_t plane[2];            // elements between two (batch, group) planes of k[i] / v[i]
    void *o;
    float *lse;
    float *po, *plse;            // decode partials [slots][B*hq][d] and [slots][B*hq]
    DevStatus *ds;
};

// One row tile and the range of keys it reads.
struct Item {
    int tok0, ntok;   // first token row (of [B*L] or, decode, of [B]) and tokens
    int g;            // KV group
    int src;          // which k / v
    int plane;        // (batch, group) plane of k / v
    int key0, nkeys;  // first key and number of keys
    int off;          // row of token i sees key j (both relative) iff j <= off + i
    int slot;         // decode: partial slot
    int split;        // the streams split the keys
    int foreign;      // the last tile of 128 keys reaches beyond this sequence's own
};

// Tokens of sequence b's own (the join kernel reports a length outside [0, cap]).
__device__ __forceinline__ int own_len(const Args &a, int b) { return min(max(a.lens[b], 0), a.cap); }

__host__ __device__ __forceinline__ int pre_items(const Args &a) { return a.hkv * a.pre_tiles * a.pre_slots; }
__host__ __device__ __forceinline__ int suf_items(const Args &a) { return a.hkv * a.B * a.suf_slots; }

__device__ __forceinline__ int item_count(const Args &a) {
    if (a.decode) return pre_items(a) + suf_items(a);
    return a.plan ? *a.plan_n * a.hkv : a.B * a.hkv * a.tiles;
}

// Item i of the call, dearest first; false when it has no rows or no keys.
__device__ __forceinline__ bool get_item(const Args &a, int i, Item &it) {
    if (!a.decode) {
        int start, len, t, b, tok = a.tok;
        if (a.plan) {
            const int4 p = a.plan[i / a.hkv];
            it.g = i % a.hkv;
            b = 0; start = p.x; len = p.y; t = p.z; it.split = p.w;
        } else {
            const int bh = i % (a.B * a.hkv);
            b = bh / a.hkv;
            it.g = bh % a.hkv;
            start = 0; len = a.L; t = (a.tiles - 1 - i / (a.B * a.hkv)) * tok; it.split = a.split;
        }
        if (a.plan && it.split) tok /= 2;
        it.tok0 = b * a.L + start + t;
        it.ntok = min(tok, len - t);
        it.src = 0;
        it.plane = b * a.hkv + it.g;
        it.key0 = start;
        it.nkeys = t + it.ntok;
        it.off = t;
        it.slot = 0;
        it.foreign = (it.nkeys + 127) / 128 * 128 > len;
        return it.ntok > 0;
    }
    it.off = kNoMask;
    it.foreign = 1;
    it.split = a.split;
    const int np = pre_items(a);
    if (i < np) {
        it.g = i % a.hkv;
        const int r = i / a.hkv, tile = r % a.pre_tiles;
        it.slot = r / a.pre_tiles;
        it.tok0 = tile * a.tok;
        it.ntok = min(a.tok, a.B - it.tok0);
        it.src = 0;
        it.plane = it.g;
        it.key0 = it.slot * a.pre_sub;
        it.nkeys = min(a.pre_sub, a.L - it.key0);
    } else {
        i -= np;
        it.g = i % a.hkv;
        const int r = i / a.hkv, s = r / a.B;
        it.tok0 = r % a.B;
        it.ntok = 1;
        it.src = 1;
        it.plane = it.tok0 * a.hkv + it.g;
        it.slot = a.pre_slots + s;
        it.key0 = s * a.suf_sub;
        it.nkeys = min(a.suf_sub, own_len(a, it.tok0) - it.key0);
    }
    return it.ntok > 0 && it.nkeys > 0;
}

// ------------------------------------------------------------------ launches
// A call's kernels run one behind the other on its stream.  Each but the first is
// launched so that its blocks may start while the kernel before it drains: it does
// its own set-up, then waits (dependency_wait, executed by every thread that reads or
// writes global memory) until that kernel is complete and its results are visible.
// A kernel lets the next one start by dependents_may_start (or by ending).
__device__ __forceinline__ void dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void dependents_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_next(bool behind_kernel, void (*kernel)(P...), int grid, int threads, size_t smem, cudaStream_t st,
                        int cluster, A &&...args) {
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((unsigned)grid);
    c.blockDim = dim3((unsigned)threads);
    c.dynamicSmemBytes = smem;
    c.stream = st;
    cudaLaunchAttribute at[2]{};
    c.attrs = at;
    if (behind_kernel) {
        at[c.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[c.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {  // (grid is a multiple of it)
        at[c.numAttrs].id = cudaLaunchAttributeClusterDimension;
        at[c.numAttrs].val.clusterDim.x = cluster;
        at[c.numAttrs].val.clusterDim.y = at[c.numAttrs].val.clusterDim.z = 1;
        ++c.numAttrs;
    }
    return cudaLaunchKernelEx(&c, kernel, std::forward<A>(args)...);
}

// ------------------------------------------------------------------ launchers
// Work lists, made on the device from the sequences' bounds: the items of a job, dearest
// first.  A cu_seqlens that does not rise inside [0, L] is reported and gives no items.
enum PlanKind {
    kRows,       // tiles of `tok` tokens
    kRowsSplit,  // the same; sequences too long for their tiles to be one SM's share of the work are
                 // cut into tiles of half as many tokens, whose two streams split the keys
    kKeys,       // tiles of `tok` keys
    kKeysSplit   // tiles of 128 keys; where more rows see a tile than key_limit allows, in pieces
};
constexpr int kPlanSms = 148;
struct PlanJob {
    int kind;
    const int32_t *cu;  // null: n_seq sequences of L tokens each
    int n_seq, L, tok, G, hkv;
    int4 *plan, *piece;  // kRows*: {first token, length, item's first token, split}; kKeys*: {.., .., tile, piece}
    int32_t *n;          // piece: {first row tile, end, partial slot of group 0 or -1, 0}
    int4 *cut;           // kKeysSplit: {first token, length, tile, slot | pieces << 16} of every cut tile
    int32_t *n_cut;
};
// A key tile whose rows are more than an SM's share of `work` steps (and an eighth, so that
// a last round of whole tiles is not cut for nothing) is cut into pieces of at most
// key_limit row tiles: two thirds of an SM's share, but worth their partials (4 steps).
// (Backward of one prompt of 2K, 4K and 8K tokens, 16 heads in 2 groups, d = 128: 91, 229 and
// 777 us; pieces of a whole share 91, 247 and 851, of half of one 87, 237 and 836; uncut 233,
// 480 and 1188.)
// A cut tile has fewer than 2 rows / limit pieces, so all cut tiles together have fewer
// than 3 kPlanSms: the number of partial slots is bounded whatever the lengths are.
__host__ __device__ __forceinline__ int key_limit(unsigned long long work) {
    const unsigned long long l = 2 * work / (3 * kPlanSms) + 1;
    return l < 4 ? 4 : l > 0x3fffffff ? 0x3fffffff : (int)l;
}
__host__ __device__ __forceinline__ bool cut_rows(int rows, unsigned long long work) {
    return rows > key_limit(work) && 8ull * kPlanSms * rows > 9ull * work;
}
constexpr int kMaxPieces = 3 * kPlanSms;
// words of the workspace header behind the status word
constexpr int kHeaderWords = (int)(kWsHeader / 4), kWordPlanN = 8, kWordKPlanN = 9, kWordCutN = 10,
              kWordNext = 32;
__device__ __forceinline__ bool header_word_of_plan(int i) { return i >= kWordPlanN && i <= kWordCutN; }
// The first of a call's launches: also zeroes the rest of the header.
cudaError_t launch_plan(const PlanJob &job0, const PlanJob *job1, DevStatus *ds, cudaStream_t st);
inline int64_t plan_cap(int L, int n_seq, int tok) { return (int64_t)L / tok + n_seq; }

struct BwdArgs {
    Args a;                      // a.plan: the row tiles; a.q, a.k, a.v as in the forward
    const int4 *kplan, *kpiece;  // the key tiles (PlanJob; else null: ktiles per batch row, uncut)
    const int32_t *kplan_n;
    int ktiles;
    const int4 *cut;             // the tiles whose rows are cut into pieces (PlanJob)
    const int32_t *n_cut;
    float *part;                 // partials of cut tiles [slot][dv, dk][128][d]
    const void *o, *dO;
    const float *lse;
    float *delta;                // [B*L, h_q]  dO . o
    void *dq, *dk, *dv;
};

// One tile of keys of the backward and the sequence whose rows read it.
struct KeyItem {
    int64_t row0;       // token row (of [B*L]) of the sequence's first token
    int start, len;     // the sequence inside its batch row
    int n0, nkeys;      // first key (of the sequence) and keys
    int g, plane;
    int j0, j1;         // tensor cores: row tiles (of 128 / G tokens) to walk
    int slot;           // partial slot, or -1: the only piece
};

__device__ __forceinline__ int key_item_count(const BwdArgs &b) {
    return b.kplan ? *b.kplan_n * b.a.hkv : b.a.B * b.a.hkv * b.ktiles;
}

// Key item i (dearest first: the first keys are read by the most rows) of tiles of `keys`.
__device__ __forceinline__ bool get_key_item(const BwdArgs &b, int i, int keys, KeyItem &it) {
    int tile, row;
    if (b.kplan) {
        const int4 p = b.kplan[i / b.a.hkv];
        it.g = i % b.a.hkv;
        row = p.x / b.a.L; it.start = p.x % b.a.L; it.len = p.y; tile = p.z;
    } else {
        const int bh = i % (b.a.B * b.a.hkv);
        row = bh / b.a.hkv;
        it.g = bh % b.a.hkv;
        it.start = 0; it.len = b.a.L; tile = i / (b.a.B * b.a.hkv);
    }
    it.row0 = (int64_t)row * b.a.L + it.start;
    it.n0 = tile * keys;
    it.nkeys = min(keys, it.len - it.n0);
    it.plane = row * b.a.hkv + it.g;
    if (b.kpiece) {
        const int4 c = b.kpiece[i / b.a.hkv];
        it.j0 = c.x;
        it.j1 = c.y;
        it.slot = c.z < 0 ? -1 : c.z + it.g;
    } else {
        const int tt = 128 / b.a.G;
        it.j0 = it.n0 / tt;
        it.j1 = (it.len + tt - 1) / tt;
        it.slot = -1;
    }
    return it.nkeys > 0;
}

// fp32, on the CUDA cores (tiles of kSimtRows rows and keys); clears the header likewise
cudaError_t launch_fwd_simt(const Args &a, int d, int64_t items, cudaStream_t st);
// bf16, on the tensor cores (decode: the prefix items): a.tok is two row tiles (128 / G tokens each), but for a
// decode call whose batch fits one; `next`: an int32 of the header for the items dealt.
// The header is cleared here where no kernel before it did (a.plan is null).
cudaError_t launch_fwd_tc(const Args &a, int d, int64_t items, int32_t *next, cudaStream_t st);
// a.tok = 128 / G, key tiles of 128; `next`: two zero int32
cudaError_t launch_bwd_tc(const BwdArgs &b, int d, int64_t row_items, int64_t key_items, int32_t *next, cudaStream_t st);
// bf16: the decode step's own caches; `first`: no kernel of the call ran before (clears the header)
cudaError_t launch_cache(const Args &a, int d, bool first, cudaStream_t st);
cudaError_t launch_combine(const Args &a, int d, bool bf16, cudaStream_t st);
cudaError_t launch_add_pieces(const BwdArgs &b, int d, cudaStream_t st);
cudaError_t launch_delta(const BwdArgs &b, int d, const int32_t *cu, int n_seq, cudaStream_t st);  // fp32
cudaError_t launch_bwd_simt(const BwdArgs &b, int d, int64_t row_items, int64_t key_items, cudaStream_t st);

}  // namespace dense
}  // namespace hsa

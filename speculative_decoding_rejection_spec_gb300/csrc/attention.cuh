// attention.cuh -- attention of a step's new tokens over the paged cache (sm_103a).
//
// For request r, kv head h and a block of up to 256 query rows (row m = new token m / G, query head
// h * G + m % G), over tiles of 128 keys:
//   S = Q K^T (tcgen05, operands in shared memory), P = exp2(S * scale * log2(e) - M) with the
//   running maximum M of each row, O = O + P V (P read from tensor memory), l = l + sum P.
//
// One block per SM, warps by role:
//   warps 0-3, 4-7  two softmax groups, a thread per row: S from tensor memory to registers, mask,
//                   maximum, exponentials, P back over S.  M only moves when a row's maximum has
//                   grown by more than 2^8 since, so the accumulator in tensor memory is rarely
//                   rescaled.  The largest P is 1 when M moves, and stays below 2^8; of fp16, whose
//                   numbers below 2^-14 lose bits and end at 2^-24, 2^7 and 2^15.
//   warps 10, 11 / 14, 15  load tiles of K / V, page by page, through TMA into a ring of slots; two
//                   warps share a tile's copies: one warp cannot issue those of small pages fast enough
//                   (a streaming loop over 16-token pages reached 3.6 TB/s with one warp issuing, 6.0
//                   with two, 6.6 with four)
//   warp 13         issues the matrix products (one thread)
//   warps 12, 8, 9  load Q; the first walks the list of work ahead of the others and announces it in
//                   a ring
// (a scheduler serves the warps of one number modulo 4: the products share theirs with no loads, and
// warps 0 and 4, which have all of the softmax's work when a row block has at most 32 rows, with none)
// A block of more than 128 rows ("wide") gives each group 128 of them and both use every tile: the
// products of one group run while the other computes its exponentials.  A block of at most 128 rows
// ("narrow": decoding and most verify steps) gives both groups the same rows and every other tile,
// merged at the end; the tiles are padded to 128 rows, which costs nothing while memory bounds the
// call (128 keys of K and V at head_dim 128 are 64 KB, 1.45 us of one SM's share of HBM bandwidth;
// their two products take 0.55 us).
//
// The work of a call is the list of all (request, head, row block, key tile), cut into equal
// contiguous shares, one per block, whatever the lengths; each row block counts as kBlockCost tiles
// more.  A (request, head, row block) that is cut leaves partial sums (O, M, l), which a second kernel
// joins.
//
// Windows (kWindow): a row block's keys are numbered without those between the sinks and the window of its first row
// (struct Range); tiles, masks and shares go by these numbers, only the lookup of pages by positions, and a tile may
// hold the last sinks and the first of the window.
// Shared prefixes (kShared): the list has for each group the row blocks of all its requests' rows together, over the
// shared tokens, without masks, and for each request those over its own tokens behind them.  A row's two results stay
// sums in the workspace and are joined by rows.
// In both, two heads of a request of at most 128 rows are taken together where both lie whole in a share ("twins"):
// a group each, over every tile of its head, nothing to merge.
//
// What bounds it (GB300; measured rates 6792 GB/s, 1923.6 TFLOP/s): decoding and verifying long
// contexts, HBM (64 requests of 1 to 8191 keys, 1.03 GB: 168 us, 6.1 TB/s, nothing read twice); short
// ones, the start of a block (the search for its share, the tables, the code itself, which comes from memory: the
// first scores are there after 6 us of one request, 11 of 64) and the join; prompt chunks, the chain of a group:
// softmax, product with V, product with the next K, as P lies over S (1700 cycles of softmax; the issuing
// thread waits 950 of some 3500 cycles per wide tile for P; the products alone take 2120: 1.3 PFLOP/s in
// the kernel).  Announcing P in two halves, so that half of its product runs beside the other half's exponentials:
// prompt chunks 304 -> 298 us, but windows over prompts 85.5 -> 88 and a shared verify step 237 -> 247; dropped.
// Windows: decoding, HBM (64 requests, window 4096, 955 MB: 162 us, 5.9 TB/s); prompt chunks (window 1024), the same
// chain (1.9 us of 128 keys and 256 rows, 1.7 where no key is hidden) and 5 us around each row block of nine tiles.
// Shared prefixes: 64 requests of one token behind two prefixes, their own tokens at HBM's rate and the start; a
// verify step (128 x 9 tokens behind four prefixes of 3 to 12 thousand), the group's wide tiles (1.7 us each).
#pragma once

#include <algorithm>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache.cuh"
#include "drain.cuh"
#include "parts.cuh"
#include "places.cuh"

namespace specrej {
namespace {

// keys per tile, and rows per softmax group.  Tiles of 64 keys with two score buffers each, so that the
// next scores run beside the exponentials, were slower everywhere (prompt chunks 0.516 ms against
// 0.330): twice the steps of the issuing thread, and products of 64 columns are bound by shared memory.
constexpr int kTile = 128;
constexpr int kBlockRows = 256;     // query rows of a (request, head, row block)
constexpr int kSoftmaxWarps = 8, kLoadWarps = 4, kMmaWarp = 13, kWalkWarp = 12, kQueryWarps = 3;
constexpr int kAttnThreads = 512;
constexpr int kSoftmaxRegs = 144, kOtherRegs = 112;  // 256 threads of each: the launch's 128 a thread in all
constexpr int kItems = 4;           // row blocks announced ahead
constexpr int kMaxGrid = 160;       // blocks a call may use (SMs of the device, 152 on GB300)
// What beginning and ending a row block costs, in tiles: without it blocks with many short contexts end
// late (0 / 2 / 4 / 6: decoding 200 / 178 / 176 / 180 us, verifying 234 / 205 / 205 / 206).
constexpr int kBlockCost = 3;
constexpr int kMinShare = 2;        // least places of a block's share (2 / 4 / 8: one token 17 / 20 / 23 us)
// Windows and shared prefixes, whose calls mix row blocks of both kinds and many of few tiles, weigh them in thirds
// of a narrow tile.  (Measured in the blocks: a narrow tile 1.05-1.3 us, a wide one 1.7-1.8; beginning and ending a
// row block 2.5-3.2 us of twins, 4.5 of a narrow one and 5.5-7 of a wide one.  Twins as narrow ones: a shared batch in
// plain decoding 59 us against 57; narrow ones as twins: windows over trees 38.9 us against 36.9.)
constexpr int kNarrowTile = 3, kWideTile = 5, kTwinBlock = 8, kNarrowBlock = 10, kWideBlock = 14;
constexpr int kMinWeighed = 7;      // as kMinShare; at least one tile's places in any case (7 / 10: one token 14.6 / 15.9)
constexpr float kLazy = 8.0f;       // log2 of the growth that moves a row's maximum (4 is no faster)
// log2 of the largest weight when a row's maximum moves.  fp16: far below the maximum, where a long context
// may have a good part of its weight, the product with V keeps 2^-21 of it in full and 2^-32 at all (with
// weights of at most 1 to 2^8 as in bf16: 2^-14 and 2^-25).
template <int DT> constexpr float kHead = DT == SPEC_F16 ? 7.0f : 0.0f;
// What the rows of a call see: their whole context; its last positions and the first ones (spec_attention_window);
// the context, of which a part is read once for several requests (spec_attention_shared).
enum Mode { kWhole, kWindow, kShared };
constexpr int kTmemColumns = 512;   // two groups: 128 of S (P over it), up to 128 of O

// A block's share of the list: [begin(x), begin(x + 1)), in tiles of cost.
struct Shares {
    int64_t each;  // the first `more` shares have one more than each
    int32_t blocks, more;
    template <int LEAST> __device__ __forceinline__ void cut(int64_t cost, int most)
    {
        if (cost < INT32_MAX) {  // nearly always: a 64-bit division takes some hundred cycles
            blocks = max(1, min(most, (int)(((uint32_t)cost + LEAST - 1) / LEAST)));
            each = (uint32_t)cost / (uint32_t)blocks;
        } else {
            blocks = most;
            each = cost / blocks;
        }
        more = (int)(cost - each * blocks);
    }
    __device__ __forceinline__ int64_t begin(int x) const { return each * x + min(x, more); }
    // the block whose share holds place t
    __device__ __forceinline__ int owner(int64_t t) const
    {
        const int64_t big = (each + 1) * more;
        if (t < INT32_MAX)
            return t < big ? (uint32_t)t / (uint32_t)(each + 1) : more + (uint32_t)(t - big) / (uint32_t)each;
        return (int)(t < big ? t / (each + 1) : more + (t - big) / each);
    }
};

struct Partial {  // of the row block that starts in a block's share and goes on behind it
    int32_t r, h, b, rows;  // rows 0: none
    int64_t last_place;     // of its last tile in the list
    Shares shares;
};

struct AttentionParams {
    const char *q, *v;  // v: the layer's values
    char *out;
    float *lse;
    int64_t q_token, q_head, out_token, out_head;  // elements
    int32_t heads, group, B;
    int32_t blocks;    // of the attention kernel
    uint32_t group_mul, group_shift;  // m / group = m * group_mul >> group_shift for 0 <= m < 2^31
    int32_t box;       // tokens per copy of K or V
    int32_t q_tokens;  // tokens of 128 query rows, when the group divides them: Q of wide row blocks then
                       // comes as one copy per 64 elements; 0: row by row
    int64_t N;
    const int32_t *cu, *parent;
    float scale_log2;
    int32_t out_by_32;  // every row of out is whole 32-byte sectors
    // workspace
    Partial *partial;   // [grid]
    float2 *part_ml;    // [grid * 2 * max_rows] M, l (0, -1: a row of a refused request, whose part_o is not written)
    float *part_o;      // [grid * 2 * max_rows * DP]
    int32_t max_rows;
    // windows
    int32_t window, sinks;
    // shared prefixes
    const int4 *shared;  // [B] first request, end, tokens of the request's group
    float2 *row_ml;      // [2][N * heads] M, l of a row over its group's tokens, over its own (as part_ml)
    float *row_o;        // [2][N * heads * DP]
    int2 *row_parts;     // [2][N * heads] of a row block, at its first row: the block it begins in, and the parts
                         // that it was cut into (0: none, the rows' sums are in row_o, or their results in out)
    int32_t *begun;      // [1] whether there is work at all (a malformed cu: none)
    int4 *requests;      // [B] query rows of a head (0: none, or an error), first row of q, tokens shared, first row of
                         // q of the group
};

template <int DT> __device__ __forceinline__ uint32_t from_float2(float a, float b)
{
    if (DT == SPEC_BF16) {
        const __nv_bfloat162 y = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&y);
    }
    const __half2 y = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&y);
}

// ---------------------------------------------------------------------------------------
// tcgen05, TMA and barriers
// ---------------------------------------------------------------------------------------

__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 columns of this thread's lane.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float *x)
{
    uint32_t *r = reinterpret_cast<uint32_t *>(x);
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
                   "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
                   "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
                   "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(addr));
}

__device__ __forceinline__ void tmem_st32(uint32_t addr, const float *x)
{
    const uint32_t *r = reinterpret_cast<const uint32_t *>(x);
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
                 "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
                 "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
                 "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
                 "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
                 "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
                 : "memory");
}

// Shared-memory matrix descriptor, 128-byte swizzle.  Rows of 128 bytes in groups of 8 (1024 bytes
// apart: the stride byte offset); `leading` is the distance between 64-element chunks of an operand
// whose contiguous dimension is not the summed one (V), and unused (16) for Q and K.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t leading)
{
    return (uint64_t)((addr & 0x3ffff) >> 4) | (uint64_t)(leading >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// Instruction descriptor: fp32 accumulator, 16-bit A and B of one type, M = 128 rows, N columns;
// b_mn: B's contiguous dimension is N.
template <int DT> __device__ __forceinline__ constexpr uint32_t mma_desc(int n, bool b_mn)
{
    return 1u << 4 | (DT == SPEC_BF16 ? 1u : 0u) << 7 | (DT == SPEC_BF16 ? 1u : 0u) << 10 | (b_mn ? 1u : 0u) << 16 |
           (uint32_t)(n >> 3) << 17 | (uint32_t)(128 >> 4) << 24;
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
                 : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
                 "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
                 : "memory");
}

// Arrives on the barrier when every product this thread has issued is done.
__device__ __forceinline__ void mma_commit(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}

// 32 bytes of one thread: a whole sector.  The rows of the threads of a warp are apart, and a store costs the memory
// pipe a cycle per row whatever it brings.
__device__ __forceinline__ void store32(void *dst, const uint32_t *x)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(x[0]), "r"(x[1]), "r"(x[2]),
                 "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t *bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ bool mbar_test_wait(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
                 : "=r"(ok)
                 : "r"(smem_addr(bar)), "r"(parity)
                 : "memory");
    return ok != 0;
}

__device__ __forceinline__ void fence_proxy_async_shared()
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap *map, int x, int token, int head, int page,
                                        uint64_t *bar)
{
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
                 "l"(map), "r"(x), "r"(token), "r"(head), "r"(page), "r"(smem_addr(bar))
                 : "memory");
}

// One lane of the (converged) warp: behind this predicate the compiler knows that a single lane is
// active and takes the operands of products and copies from uniform registers.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
    return p != 0;
}

// A row block of this block's share, as the roles need it.  nt = 0 ends the share.
struct alignas(16) Item {
    int32_t r, h, b;       // request, kv head, row block
    int32_t rows, nt;      // query rows; tiles in the share
    int32_t t0, tiles;     // the first of those, and tiles of the row block
    int32_t keys;          // keys up to the last row's own
    int32_t len, n, first; // of the request: committed tokens, new tokens, its first row
    int32_t q_use;         // Q slots used before (a narrow row block takes one, a wide one both)
    uint32_t slots;        // K / V slots used before
    int32_t near, gap;     // as Range's; keys and len are without those left out
    int32_t kind;          // 0: the result goes to out; 1: it is that over a group's shared tokens (the rows are
                           // those of all its requests); 2: that over the other tokens of a request of a group;
                           // 4 more: twins, the same of head h + 1 with it, a group each
};

__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap *map, int x, int head, int token, uint64_t *bar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
                 "l"(map), "r"(x), "r"(head), "r"(token), "r"(smem_addr(bar))
                 : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

__device__ __forceinline__ void copy16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void zero16(uint32_t dst)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(dst), "r"(0) : "memory");
}

// What a block keeps behind the operand tiles.
template <int SLOTS> struct alignas(16) AttnShared {
    // per group: (M, l) of its rows at the end of a narrow row block, or a tree's parents at its start
    union {
        float2 ml[kTile];
        int32_t parent[kMaxTree];
    } group[2];
    Item item[kItems];
    uint64_t full[SLOTS], empty[SLOTS];  // a slot's tile has landed / has been used
    uint64_t s_full[2], p_full[2], o_full[2];  // a group's S is there / its P / the last of its O
    uint64_t q_full[2], q_empty[2];      // a slot's Q is there / has been used
    uint64_t item_full[kItems], item_empty[kItems];
    uint64_t ready, merge, done;
    uint64_t known[2];  // group 0 of a wide row block has looked at its last values (by turns)
    uint32_t tmem;
    uint32_t arrivals[SLOTS + 2];  // made on full[] and q_full[] in all, added up as the loading roles end
    volatile int32_t gave_up;
    // the number of a row block among those with unseen keys, by its last bit (of twins, by group)
    volatile int32_t spoilt[2][2];
};

// Waits for a barrier's phase, a bounded number of polls.  When one wait gives up, all do: no row block
// is begun, no copy started and no slot given back any more; the softmax of what has begun runs through
// without waiting (its indices are those of an announced row block); the roles leave together, and the
// copies in flight are waited for before the block does.  A wait of try_wait is suspended and
// woken late; the thread that issues the products polls instead (SPIN): prompt chunks 0.356 -> 0.330 ms.
// The others do not, for the sake of the schedulers they share.
template <bool SPIN>
__device__ __forceinline__ bool attn_wait(uint64_t *bar, uint32_t parity, volatile int32_t *gave_up, int32_t *error)
{
    for (uint32_t i = 0; i < (SPIN ? 64 * kWaitLimit : kWaitLimit); ++i) {
        if (SPIN ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity))
            return true;
        if ((!SPIN || i % 64 == 63) && *gave_up)
            return false;
    }
    *gave_up = 1;
    atomicOr(error, SPEC_DEVERR_TIMEOUT);
    return false;
}

__device__ __forceinline__ int by_group(const AttentionParams &p, int m)
{
    return (int)((uint64_t)(uint32_t)m * p.group_mul >> p.group_shift);
}

// ---------------------------------------------------------------------------------------
// The list of work
// ---------------------------------------------------------------------------------------

struct Request {
    int n, len, rows;  // new tokens, committed tokens, query rows
    int cost;          // of all its row blocks (one head), in tiles
    // of a request in a group: the tokens that it shares (0: no group); of the first request of one, the query
    // rows of the group and the cost of their row blocks, which stand before its own in the list
    int tokens, group_rows, group_cost;
};

// The keys of a row block, numbered without those that none of its rows sees: the first `near` are the request's
// first, `gap` are left out behind them, and there are `keys` in all.  Tiles, masks and lengths go by these numbers,
// only the lookup of pages by positions.
struct Range {
    int keys, near, gap;
    __device__ __forceinline__ int tiles() const { return (keys + kTile - 1) / kTile; }
};

// The places of a row block in the list: `begin`, then `tile` for each tile, done by the block whose share has the
// first of them.
struct Cost {
    int begin, tile;
    __device__ __forceinline__ int of(int tiles) const { return begin + tile * tiles; }
    // the first tile whose first place is `at` or behind it
    __device__ __forceinline__ int first(int at) const
    {
        return at <= begin ? 0 : (uint32_t)(at - begin + tile - 1) / (uint32_t)tile;
    }
};

// ... of a block of `rows` of all the rows of a request or group
template <int MODE> __device__ __forceinline__ Cost cost_of(const AttentionParams &p, int rows, int all)
{
    if (MODE == kWhole)
        return Cost{kBlockCost, 1};
    if (rows > kTile)
        return Cost{kWideBlock, kWideTile};
    return Cost{all <= kTile && p.heads > p.group ? kTwinBlock : kNarrowBlock, kNarrowTile};
}

// Of row block b: up to the last row's own key.  What is left out begins and ends with a copy of `box` keys: before
// the window of the block's first row (the root of a tree: the others are deeper), behind the sinks; or the tokens of
// the group.
template <int MODE>
__device__ __forceinline__ Range block_range(const AttentionParams &p, const Request &q, bool of_group, int b)
{
    if (MODE == kShared && of_group)
        return Range{q.tokens, 0, 0};
    const int end = min((b + 1) * kBlockRows, q.rows);
    Range x{q.len + by_group(p, end - 1) + 1, 0, MODE == kShared ? q.tokens : 0};
    if (MODE == kWindow) {
        const int low = q.len + (p.parent ? 0 : by_group(p, b * kBlockRows)) - p.window + 1;
        const int from = max(low, 0) & -p.box, near = (p.sinks + p.box - 1) & -p.box;
        if (from > near) {
            x.near = near;
            x.gap = from - near;
        }
    }
    if (MODE != kWhole)
        x.keys -= x.gap;
    return x;
}

// The shared tokens of request r's group, whose entry of the plan is g, when that fits the requests as they are;
// of the first request, the group's query rows.
__device__ __forceinline__ int group_tokens(const CacheView &c, const AttentionParams &p, int r, int len, int4 g,
                                            int *rows)
{
    if (g.z <= 0 || g.z > len || g.x < 0 || g.x > r || g.y <= r || g.y > p.B || g.y - g.x < 2 || g.z % c.page_size)
        return 0;
    // (asked for together: this is part of the chain of loads that every block begins with)
    const int4 first = p.shared[g.x];
    const int first_len = c.lens[g.x], first_held = c.held[g.x], from = p.cu[g.x], to = p.cu[g.y];
    const int64_t all = ((int64_t)to - from) * p.group;
    const bool fits = (first.x == g.x) & (first.y == g.y) & (first.z == g.z) & (first_len >= g.z) &
                      holds(c, first_held, first_len, 0) & (all > 0) & (all <= p.N * p.group);
    if (!fits || (all + kBlockRows - 1) / kBlockRows * (kWideBlock + kWideTile * (1 + (int64_t)g.z / kTile)) > INT32_MAX / 2)
        return 0;
    *rows = g.x == r ? (int)all : 0;
    return g.z;
}

// The request's sizes; costs of 0 when there is nothing to do, or an error, which is recorded on demand.
template <int MODE>
__device__ __forceinline__ Request request_of(const CacheView &c, const AttentionParams &p, int r, int n, int len,
                                              int held, int4 g, bool report)
{
    Request q;
    q.n = n;
    q.len = len;
    q.rows = n * p.group;
    q.cost = q.tokens = q.group_rows = q.group_cost = 0;
    if (MODE == kShared) {
        q.tokens = group_tokens(c, p, r, len, g, &q.group_rows);
        if (q.group_rows > 0) {
            const int tiles = block_range<MODE>(p, q, true, 0).tiles(), last = q.group_rows % kBlockRows;
            q.group_cost = q.group_rows / kBlockRows * cost_of<MODE>(p, kBlockRows, q.group_rows).of(tiles) +
                           (last > 0 ? cost_of<MODE>(p, last, q.group_rows).of(tiles) : 0);
        }
    }
    if (n <= 0)
        return q;
    int64_t keys = (int64_t)len + n - (MODE == kShared ? q.tokens : 0);  // of a row block, at most
    if (MODE == kWindow)
        keys = most_window_keys(keys, p.parent ? n : min(n, by_group(p, kBlockRows) + 2), p.window, p.sinks, p.box);
    if (!holds(c, held, len, n) || (p.parent && n > kMaxTree) ||
        most_places((q.rows + kBlockRows - 1) / kBlockRows, keys, MODE == kWhole ? kBlockCost : kWideBlock,
                    MODE == kWhole ? 1 : kWideTile, kTile) > INT32_MAX) {
        if (report)
            cache_error(c.error, p.parent && n > kMaxTree ? SPEC_DEVERR_TREE : SPEC_DEVERR_LENGTH, r);
        return q;
    }
#pragma unroll 1
    for (int b = 0; b * kBlockRows < q.rows; ++b)
        q.cost += cost_of<MODE>(p, min(kBlockRows, q.rows - b * kBlockRows), q.rows)
                      .of(block_range<MODE>(p, q, false, b).tiles());
    return q;
}

template <int MODE>
__device__ __forceinline__ Request request_of(const CacheView &c, const AttentionParams &p, int r, bool report)
{
    return request_of<MODE>(c, p, r, p.cu[r + 1] - p.cu[r], c.lens[r], c.held[r],
                            MODE == kShared ? p.shared[r] : int4{}, report);
}

// Walks a block's share, one (request or group, head, row block) at a time; a whole warp.  A row block takes
// some places of the list before those of its tiles; a share that ends within them leaves the row block to the next.
// (A share has at least a tile's places, with kMinWeighed at least the 5 of a wide one from lists of 11 places on, the
// shortest there are; so it has the first place of some tile, and a row block that is cut has a part in each block from
// its first to its last.)
template <int MODE> struct Walk {
    Request q;
    int r, h, b;
    bool of_group;    // the row blocks of the group that begins with the request
    Range range;      // of this row block
    int tiles;        // of this row block
    int t0, t1;       // those in the share; t1 > t0 but for a share of no tile
    bool twins;       // with the same of the next head
    int64_t pos, end; // place in the list behind the row block's part
    int64_t last;     // place of the row block's last tile

    // r and q are the request in which the share begins, after `base` places; false when it holds no tile
    __device__ __forceinline__ bool start(const CacheView &c, const AttentionParams &p, const Shares &s, int64_t base)
    {
        pos = s.begin(blockIdx.x);
        end = s.begin(blockIdx.x + 1);
        int64_t at = pos - base;
        of_group = MODE == kShared && at < (int64_t)q.group_cost * c.heads;
        if (MODE == kShared && !of_group)
            at -= (int64_t)q.group_cost * c.heads;
        const int cost = of_group ? q.group_cost : q.cost;
        for (h = 0; at >= cost; ++h)
            at -= cost;
        for (b = 0;; ++b) {
            const int all = cost_of<MODE>(p, rows(), all_rows()).of(block_range<MODE>(p, q, of_group, b).tiles());
            if (at < all)
                break;
            at -= all;
        }
        return here(c, p, (int)at);
    }
    // the part of the row block from its place `from` on
    __device__ __forceinline__ bool here(const CacheView &c, const AttentionParams &p, int from)
    {
        range = block_range<MODE>(p, q, of_group, b);
        tiles = range.tiles();
        const Cost cost = cost_of<MODE>(p, rows(), all_rows());
        const int all = cost.of(tiles), to = (int)min((int64_t)all, from + (end - pos));
        t0 = cost.first(from);
        t1 = cost.first(to);
        last = pos - from + cost.of(tiles - 1);
        pos += to - from;
        // Two heads of few rows, both whole: a softmax group takes each, nothing is to be merged, and the one's first
        // and last steps run beside the other's.
        twins = MODE != kWhole && t0 == 0 && to == all && all_rows() <= kTile && h + 1 < c.heads && end - pos >= all;
        if (twins) {
            pos += all;
            ++h;
        }
        return t1 > t0;
    }
    // to the next row block; false at the share's end
    __device__ __forceinline__ bool next(const CacheView &c, const AttentionParams &p)
    {
        if (pos >= end)
            return false;
        if (++b * kBlockRows >= all_rows()) {
            b = 0;
            if (++h == c.heads) {
                h = 0;
                if (MODE == kShared && of_group && q.cost > 0) {
                    of_group = false;
                    return here(c, p, 0);
                }
                const int lane = threadIdx.x & 31;
                for (++r;; r += 32) {
                    bool some = false;
                    if (r + lane < p.B) {
                        const Request x = request_of<MODE>(c, p, r + lane, false);
                        some = x.cost > 0 || x.group_cost > 0;
                    }
                    const unsigned any = __ballot_sync(kFull, some);
                    if (any) {
                        r += __ffs(any) - 1;
                        break;
                    }
                    if (r >= p.B)
                        return false;  // cannot be: the share ends before
                }
                q = request_of<MODE>(c, p, r, false);
                of_group = MODE == kShared && q.group_cost > 0;
            }
        }
        return here(c, p, 0);
    }
    __device__ __forceinline__ int all_rows() const { return of_group ? q.group_rows : q.rows; }
    __device__ __forceinline__ int rows() const { return min(kBlockRows, all_rows() - b * kBlockRows); }
    __device__ __forceinline__ int kind() const { return MODE != kShared || !q.tokens ? 0 : of_group ? 1 : 2; }
    __device__ __forceinline__ int first_head() const { return h - (MODE != kWhole && twins); }
};

// ---------------------------------------------------------------------------------------
// The kernel
// ---------------------------------------------------------------------------------------

template <int DP> struct AttnSizes {
    static constexpr int kSlotBytes = kTile * DP * 2;     // a tile of K or V; a group's Q
    static constexpr int kSlots = (224 * 1024 - 2 * kSlotBytes) / kSlotBytes;  // 5 of 32 KB, 12 of 16 KB
    static constexpr int kChunk = kTile * 128;            // 64 elements of every row of a tile
    using Shared = AttnShared<kSlots>;
    static constexpr int kBytes = (2 + kSlots) * kSlotBytes + (int)sizeof(Shared);
};
static_assert(AttnSizes<128>::kBytes <= 227 * 1024 && AttnSizes<64>::kBytes <= 227 * 1024, "shared memory of one SM");

// Which of the 32 columns from `column` on row i sees: of the chain, or by the tree's bits.
__device__ __forceinline__ uint32_t low_bits(int k) { return k <= 0 ? 0u : k >= 32 ? ~0u : (1u << k) - 1; }

__device__ __forceinline__ uint32_t tree_columns(const uint32_t *bits, int len, int column)
{
    const int o = column - len;  // node of the first column
    uint32_t lo = 0, hi = 0;
#pragma unroll
    for (int j = 0; j < kMaxTree / 32; ++j) {
        lo = o >= 0 && o / 32 == j ? bits[j] : lo;
        hi = o >= 0 && o / 32 + 1 == j ? bits[j] : hi;
    }
    if (o >= 0)
        return __funnelshift_r(lo, hi, o & 31);
    return low_bits(-o) | (o > -32 ? bits[0] << -o : 0u);
}

// Two 16-bit values: bits 15 and 31 are set where they are not finite (the exponent is all ones, and one
// more carries out of it).
template <int DT> __device__ __forceinline__ uint32_t not_finite(uint32_t x)
{
    constexpr uint32_t e = DT == SPEC_BF16 ? 0x7f807f80 : 0x7c007c00;
    return (x & e) + (DT == SPEC_BF16 ? 0x00800080 : 0x04000400);
}

// Rows of V in shared memory, a thread's 16-byte units from i0 to i1 (every kTile-th): values that are not
// finite become zeros.  (Called, not inlined: prompt chunks 319 -> 324 us.)
template <int DT, int DP> __device__ __forceinline__ void drop_not_finite(char *base, int i0, int i1)
{
    for (int j = 0; j < DP / 64; ++j)
        for (int i = i0; i < i1; i += kTile) {
            uint32_t *at = reinterpret_cast<uint32_t *>(base + j * AttnSizes<DP>::kChunk + i * 16);
            for (int e = 0; e < 4; ++e) {
                const uint32_t x = at[e], bad = not_finite<DT>(x);
                at[e] = (bad & 0x8000u ? 0 : x & 0xffffu) | (bad & 0x80000000u ? 0 : x & 0xffff0000u);
            }
        }
}

// The values that are not finite among the keys [from, to) that a row sees, added to its result (a row
// of 16-bit outputs, or of fp32 partial sums).
template <int DT, int MODE>
__device__ __noinline__ void add_spoilt(const CacheView &c, const AttentionParams &p, int r, int h, int from, int to,
                                        int near, int gap, int len, int token, int low, uint4 tree, char *result,
                                        bool fp32)
{
    using T = typename std::conditional<DT == SPEC_BF16, __nv_bfloat16, __half>::type;
    const uint32_t bits[4] = {tree.x, tree.y, tree.z, tree.w};
    for (int key = from; key < to; ++key) {
        const int o = key - len;
        bool seen = p.parent ? o < 0 || (o < kMaxTree && bits[o >> 5 & 3] >> (o & 31) & 1) : o <= token;
        if (MODE == kWindow)
            seen &= key < p.sinks || key >= low;
        const int at = MODE == kWhole || key < near ? key : key + gap;
        const int place = at / c.page_size, page = seen ? c.table[r * c.table_stride + place] : -1;
        if (page < 0 || page >= c.num_pages)
            continue;
        const T *v = reinterpret_cast<const T *>(p.v) + page * c.page_stride +
                     (int64_t)(at - place * c.page_size) * c.token_stride + h * c.head_stride;
        for (int e = 0; e < c.dim; ++e) {
            const float x = (float)v[e];
            if (fabsf(x) < INFINITY)
                continue;
            if (fp32)
                reinterpret_cast<float *>(result)[e] += x;
            else
                reinterpret_cast<T *>(result)[e] = (T)((float)reinterpret_cast<T *>(result)[e] + x);
        }
    }
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Two fp32 values in one instruction.
__device__ __forceinline__ uint64_t pack2(float a, float b)
{
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ void unpack2(uint64_t x, float &a, float &b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// The shares of the list, and the request in which this block's begins (w->r and w->q, with the work
// before it); a whole warp, a request per lane.  False when the block has no share, or cu is malformed.
template <int MODE>
__device__ __forceinline__ bool find_share(const CacheView &c, const AttentionParams &p, Shares *shares,
                                           Walk<MODE> *w, int64_t *base, int lane)
{
    // Twice: the total makes the shares, then the block looks again at the 32 requests in which its own begins (lane i
    // keeps what lies before those of turn i; batches of more than 32 turns are gone through again).  The next turn's
    // loads are on their way while one is added up.
    struct Loads {
        int32_t here, next, len, held;
        int4 g;
    };
    auto load = [&](int r0) {
        const int r = min(r0 + lane, p.B - 1);
        return Loads{p.cu[min(r0 + lane, p.B)], p.cu[min(r0 + lane + 1, p.B)], c.lens[r], c.held[r],
                     MODE == kShared ? p.shared[r] : int4{}};
    };
    int64_t before = 0, at = 0, work = 0, kept = 0;
    Request q{};
    bool bad = false, wrong = false;
    auto add_up = [&](int r0, const Loads &x) {
        const int r = r0 + lane;
        bad |= x.here > x.next || x.next > p.N || x.here < 0 || (r == 0 && x.here != 0);
        q.cost = q.group_cost = q.tokens = 0;
        if (r < p.B && !bad) {
            q = request_of<MODE>(c, p, r, x.next - x.here, x.len, x.held, x.g, false);
            wrong |= q.cost == 0 && q.n > 0;
        }
        if (MODE == kShared && blockIdx.x == 0 && r < p.B)
            p.requests[r] = make_int4(q.cost > 0 ? q.rows : 0, x.here, q.tokens, q.tokens ? p.cu[x.g.x] : 0);
        work = (int64_t)q.cost * c.heads;
        if (MODE == kShared)
            work += (int64_t)q.group_cost * c.heads;
        int64_t incl = work;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t y = __shfl_up_sync(kFull, incl, d);
            incl += lane >= d ? y : 0;
        }
        at = before + incl - work;
        before += __shfl_sync(kFull, incl, 31);
    };
    Loads ahead = load(0);
#pragma unroll 1
    for (int r0 = 0; r0 < p.B; r0 += 32) {
        const Loads x = ahead;
        if (r0 + 32 < p.B)
            ahead = load(r0 + 32);
        kept = r0 == 32 * lane ? before : kept;
        add_up(r0, x);
    }
    if (__any_sync(kFull, bad)) {
        if (blockIdx.x == 0 && lane == 0)
            cache_error(c.error, SPEC_DEVERR_LAYOUT, -1);
        return false;
    }
    if (blockIdx.x == 0 && __any_sync(kFull, wrong))
        for (int r = lane; r < p.B; r += 32)
            request_of<MODE>(c, p, r, true);
    shares->template cut<MODE == kWhole ? kMinShare : kMinWeighed>(before, gridDim.x);
    if (before == 0 || blockIdx.x >= shares->blocks)
        return false;
    const int64_t want = shares->begin(blockIdx.x);
    int r0 = 0;
    if (p.B > 32) {
        const int turn = __popc(__ballot_sync(kFull, 32 * lane < p.B && kept <= want)) - 1;
        r0 = 32 * turn;
        before = __shfl_sync(kFull, kept, turn);
        add_up(r0, load(r0));
    }
#pragma unroll 1
    while (true) {
        const unsigned who = __ballot_sync(kFull, at <= want && want < at + work);
        if (who) {
            const int from = __ffs(who) - 1;
            w->r = r0 + from;
            w->q.n = __shfl_sync(kFull, q.n, from);
            w->q.len = __shfl_sync(kFull, q.len, from);
            w->q.cost = __shfl_sync(kFull, q.cost, from);
            w->q.rows = w->q.n * p.group;
            if (MODE == kShared) {
                w->q.tokens = __shfl_sync(kFull, q.tokens, from);
                w->q.group_rows = __shfl_sync(kFull, q.group_rows, from);
                w->q.group_cost = __shfl_sync(kFull, q.group_cost, from);
            }
            *base = __shfl_sync(kFull, at, from);
            return true;
        }
        r0 += 32;
        if (r0 >= p.B)
            return false;  // cannot be: every place belongs to a request
        add_up(r0, load(r0));
    }
}

// The order of a row block's tiles in the ring, as the products use them: K of tile 0, then K of tile t + 1 and V of
// tile t.  Twins: of both in every step.
__device__ __forceinline__ uint32_t slot_of(bool is_v, bool twins, int g, int t, int nt)
{
    if (twins)
        return is_v ? (t + 1 < nt ? 4 * t + 3 + 2 * g : 4 * nt - 2 + g) : (t > 0 ? 4 * t - 2 + 2 * g : g);
    return is_v ? min(2 * t + 2, 2 * nt - 1) : max(2 * t - 1, 0);
}

template <int DT, int DP, int MODE>
__global__ void __launch_bounds__(kAttnThreads, 1)
    attention_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                     const __grid_constant__ CUtensorMap qmap, CacheView c, AttentionParams p)
{
    using Z = AttnSizes<DP>;
    constexpr int SLOTS = Z::kSlots;
    extern __shared__ __align__(1024) char smem[];
    char *const qtile = smem, *const ring = smem + 2 * Z::kSlotBytes;
    auto &S = *reinterpret_cast<typename Z::Shared *>(smem + (2 + SLOTS) * Z::kSlotBytes);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    if (tid == 0) {
        prefetch_map(&kmap);
        prefetch_map(&vmap);
        if (p.q_tokens)
            prefetch_map(&qmap);
    }
    if (tid == 0) {
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(&S.full[i], 2);
            mbar_init(&S.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&S.s_full[i], 1);
            mbar_init(&S.p_full[i], 4);
            mbar_init(&S.o_full[i], 1);
            mbar_init(&S.q_full[i], kQueryWarps);
            mbar_init(&S.q_empty[i], 1);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&S.item_full[i], 1);
            mbar_init(&S.item_empty[i], kSoftmaxWarps + kLoadWarps + 1 + kQueryWarps - 1);  // all but the writer
        }
        mbar_init(&S.ready, kSoftmaxWarps);
        mbar_init(&S.merge, kSoftmaxWarps);
        mbar_init(&S.done, 1);
        mbar_init(&S.known[0], 4);
        mbar_init(&S.known[1], 4);
        for (int i = 0; i < SLOTS + 2; ++i)
            S.arrivals[i] = 0;
        S.gave_up = 0;
        S.spoilt[0][0] = S.spoilt[0][1] = S.spoilt[1][0] = S.spoilt[1][1] = 0;
        mbar_fence_init();
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&S.tmem)),
                     "r"(kTmemColumns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = S.tmem;
    auto wait = [&](uint64_t *bar, uint32_t parity) { return attn_wait<false>(bar, parity, &S.gave_up, c.error); };
    auto spin = [&](uint64_t *bar, uint32_t parity) { return attn_wait<true>(bar, parity, &S.gave_up, c.error); };

    // Waits for the row block announced as number k (in S.item[k % kItems]); the caller gives the entry
    // back with done_with() when it has read it.
    auto announced = [&](uint32_t k) { return wait(&S.item_full[k % kItems], k / kItems & 1); };
    auto done_with = [&](uint32_t k) {
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&S.item_empty[k % kItems]);
    };

    // A warpgroup sets its registers together; the roles that follow are compiled for that number.
    if (warp >= kSoftmaxWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp & 2) {
            const bool is_v = warp >= 14;
            const int half = warp & 1;  // copies (piece, chunk) of every second number
            const CUtensorMap *map = is_v ? &vmap : &kmap;
            const int pieces = kTile / p.box;
            // Copies of 32 pieces, one per lane; token < 0: behind the last key.
            struct Pieces {
                int page, token;
            };
            uint32_t arrivals = 0;  // lane i: on full[i]
            bool lost = false;
            for (uint32_t k = 0;; ++k) {
                if (!announced(k))
                    break;
                const Item &item = S.item[k % kItems];
                const int r = item.r, h = item.h, keys = item.keys, t0 = item.t0, nt = item.nt;
                const uint32_t slots = item.slots;
                const int near = item.near, gap = item.gap, heads = MODE != kWhole && item.kind & 4 ? 2 : 1;
                done_with(k);
                if (nt == 0)
                    break;
                const int32_t *row = c.table + r * c.table_stride;
                const int end = min(keys, (t0 + nt) * kTile);
                // the pieces from number 32 * i of the share's part; looked at 32 pieces later
                auto lookup = [&](int i) {
                    Pieces x{-1, -1};
                    int at = t0 * kTile + (i * 32 + lane) * p.box;
                    if (at < end) {
                        if (MODE != kWhole && at >= near)
                            at += gap;
                        const int column = at / c.page_size;
                        x.page = row[column];
                        x.token = at - column * c.page_size;
                    }
                    return x;
                };
                const int per = 32 / pieces;  // tiles of 32 pieces
                Pieces now{-1, -1}, ahead = lookup(0);
                for (int t = 0; t < nt; ++t) {
                    const int from = t % per * pieces;
                    if (from == 0) {
                        now = ahead;
                        ahead = lookup(t / per + 1);
                        if (now.token >= 0 && (now.page < 0 || now.page >= c.num_pages)) {
                            cache_error(c.error, SPEC_DEVERR_PAGE, r);
                            now.page = c.num_pages;  // outside the tensor: reads as zeros
                        }
                    }
                    for (int g = 0; g < heads; ++g) {
                        const uint32_t use = slots + slot_of(is_v, heads == 2, g, t, nt);
                        const uint32_t slot = use % SLOTS, turn = use / SLOTS;
                        const int count = __popc(__ballot_sync(kFull, now.token >= 0) >> from & low_bits(pieces));
                        if (turn > 0)
                            wait(&S.empty[slot], (turn & 1) ^ 1);
                        if (__any_sync(kFull, S.gave_up)) {
                            lost = true;
                            break;
                        }
                        arrivals += lane == slot;
                        const uint32_t dst = smem_addr(ring) + slot * Z::kSlotBytes;
                        uint64_t *bar = &S.full[slot];
                        constexpr int kChunks = DP / 64;
                        const int mine = kChunks == 2 ? count : (count + 1 - half) / 2;
                        if (elect_one())
                            mbar_arrive_expect_tx(bar, mine * p.box * 128);
                        for (int i = 0; i < mine; ++i) {
                            const int piece = kChunks == 2 ? i : 2 * i + half, chunk = kChunks == 2 ? half : 0;
                            const int page = __shfl_sync(kFull, now.page, from + piece);
                            const int token = __shfl_sync(kFull, now.token, from + piece);
                            if (elect_one())
                                tma_box(dst + piece * p.box * 128 + chunk * Z::kChunk, map, chunk * 64, token, h + g, page,
                                        bar);
                        }
                        __syncwarp();
                    }
                    if (lost)
                        break;
                }
            }
            if (lane < SLOTS)
                atomicAdd(&S.arrivals[lane], arrivals);
        } else if (warp == kMmaWarp) {
            if (elect_one()) {
                const uint64_t q_desc = smem_desc(smem_addr(qtile), 16), k_desc = smem_desc(smem_addr(ring), 16),
                               v_desc = smem_desc(smem_addr(ring), Z::kChunk);
                // A wait costs this thread some 200 cycles even when there is nothing to wait for, and it has
                // to stay ahead of the products it has issued (about seven fit the queue, 500 cycles): the
                // barriers of the next step are looked at together, beside the commits of this one, and
                // waited for only if they were not through then.
                uint32_t slot = 0, turn = 0, p_turn = 0;  // p_turn: a bit per group
                bool lost = false;                        // a wait gave up: no slot is given back any more
                auto full_here = [&](uint32_t i) {        // slot i from the next
                    const uint32_t s = slot + i;
                    return s < SLOTS ? mbar_test_wait(&S.full[s], turn) : mbar_test_wait(&S.full[s - SLOTS], turn ^ 1);
                };
                auto take = [&](bool here) {  // the next slot, landed
                    if (!here)
                        lost |= !spin(&S.full[slot], turn);
                    const uint32_t s = slot;
                    if (++slot == SLOTS) {
                        slot = 0;
                        turn ^= 1;
                    }
                    return s;
                };
                auto scores = [&](int g, uint32_t kslot, int qslot) {
                    const uint64_t a = q_desc + qslot * (Z::kSlotBytes >> 4), b = k_desc + kslot * (Z::kSlotBytes >> 4);
#pragma unroll
                    for (int i = 0; i < DP / 16; ++i) {
                        const uint32_t o = (i / 4 * Z::kChunk + i % 4 * 32) >> 4;
                        mma_ss(tmem + g * 256, a + o, b + o, mma_desc<DT>(kTile, false), i > 0);
                    }
                };
                auto outputs = [&](int g, uint32_t vslot, bool add) {
                    const uint64_t b = v_desc + vslot * (Z::kSlotBytes >> 4);
#pragma unroll
                    for (int i = 0; i < kTile / 16; ++i)
                        mma_ts(tmem + g * 256 + kTile, tmem + g * 256 + i * 8, b + (i * 2048 >> 4),
                               mma_desc<DT>(DP, true), i > 0 || add);
                };
                auto p_here = [&](int g) { return mbar_test_wait(&S.p_full[g], p_turn >> g & 1); };
                auto p_ready = [&](int g, bool here) {
                    if (!here)
                        lost |= !spin(&S.p_full[g], p_turn >> g & 1);
                    p_turn ^= 1u << g;
                    tmem_fence_after();
                };
                lost = !wait(&S.ready, 0);
                for (uint32_t k = 0; !lost; ++k) {
                    if (!announced(k))
                        break;
                    const Item &item = S.item[k % kItems];
                    const int nt = item.nt, q_use = item.q_use;
                    const bool wide = item.rows > kTile, twins = MODE != kWhole && item.kind & 4;
                    mbar_arrive(&S.item_empty[k % kItems]);
                    if (nt == 0)
                        break;
                    for (int g = 0; g <= (int)(wide || twins); ++g)
                        lost |= !wait(&S.q_full[(q_use + g) & 1], (q_use + g) >> 1 & 1);
                    // step t: scores of tile t, outputs of tile t - 1
                    bool k_in = false, v_in = false, p_in = false;
                    if (MODE != kWhole && twins) {
                        for (int t = 0; t <= nt && !lost; ++t) {
#pragma unroll 1
                            for (int g = 0; g < 2; ++g) {
                                uint32_t kslot = 0, vslot = 0;
                                if (t < nt)
                                    kslot = take(k_in);
                                if (t > 0) {
                                    vslot = take(v_in);
                                    p_ready(g, p_in);
                                    outputs(g, vslot, t > 1);
                                }
                                if (t < nt)
                                    scores(g, kslot, (q_use + g) & 1);
                                mma_commit(t < nt ? &S.s_full[g] : &S.o_full[g]);
                                if (lost)
                                    break;
                                // the next half step's: K where there is one, V behind it, and the group's weights
                                const int nextt = t + g;
                                k_in = nextt < nt && full_here(0);
                                v_in = nextt > 0 && nextt <= nt && full_here(nextt < nt);
                                p_in = nextt > 0 && nextt <= nt && p_here(g ^ 1);
                                if (t < nt) {
                                    mma_commit(&S.empty[kslot]);
                                    if (t + 1 == nt)
                                        mma_commit(&S.q_empty[(q_use + g) & 1]);
                                }
                                if (t > 0)
                                    mma_commit(&S.empty[vslot]);
                            }
                        }
                    } else if (!wide) {
                        for (int t = 0; t <= nt; ++t) {
                            const int g = (t - 1) & 1;  // the group of tile t - 1
                            uint32_t kslot = 0, vslot = 0;
                            if (t < nt) {
                                kslot = take(k_in);
                                scores(t & 1, kslot, q_use & 1);
                                mma_commit(&S.s_full[t & 1]);
                            }
                            if (t > 0) {
                                vslot = take(v_in);
                                p_ready(g, p_in);
                                outputs(g, vslot, t > 2);
                                if (t + 1 >= nt)
                                    mma_commit(&S.o_full[g]);
                            }
                            if (lost)
                                break;
                            if (t < nt) {
                                const bool more = t + 1 < nt;
                                k_in = more && full_here(0);
                                v_in = full_here(more);
                                p_in = p_here(t & 1);
                                mma_commit(&S.empty[kslot]);
                                if (!more)
                                    mma_commit(&S.q_empty[q_use & 1]);
                            }
                            if (t > 0)
                                mma_commit(&S.empty[vslot]);
                        }
                    } else {
                        for (int t = 0; t <= nt; ++t) {
                            uint32_t kslot = 0, vslot = 0;
                            if (t < nt)
                                kslot = take(k_in);
                            if (t > 0)
                                vslot = take(v_in);
#pragma unroll
                            for (int g = 0; g < 2; ++g) {
                                if (t > 0) {
                                    p_ready(g, g == 0 && p_in);
                                    outputs(g, vslot, t > 1);
                                }
                                if (t < nt)
                                    scores(g, kslot, (q_use + g) & 1);
                                mma_commit(t < nt ? &S.s_full[g] : &S.o_full[g]);
                            }
                            if (lost)
                                break;
                            if (t < nt) {
                                const bool more = t + 1 < nt;
                                k_in = more && full_here(0);
                                v_in = full_here(more);
                                p_in = p_here(0);
                                mma_commit(&S.empty[kslot]);
                                if (!more) {
                                    mma_commit(&S.q_empty[0]);
                                    mma_commit(&S.q_empty[1]);
                                }
                            }
                            if (t > 0)
                                mma_commit(&S.empty[vslot]);
                        }
                    }
                }
                // every product is done before the block gives its memory back
                mma_commit(&S.done);
                for (uint32_t i = 0; i < kWaitLimit && !mbar_try_wait(&S.done, 0); ++i) {
                }
            }
            __syncwarp();
        } else {
            Walk<MODE> w;
            Shares shares;
            const int part = warp == kWalkWarp ? 0 : warp - 7;
            int q_use = 0;
            uint32_t slots = 0, arrivals = 0;  // arrivals: lane i: on q_full[i]
            bool more = false;
            if (warp == kWalkWarp) {
                if (lane == 0)
                    p.partial[blockIdx.x].rows = 0;
                int64_t base;
                const bool found = find_share(c, p, &shares, &w, &base, lane);
                if (MODE == kShared && blockIdx.x == 0 && lane == 0)
                    *p.begun = found;  // of the first block: whenever there is any work
                more = found && (w.start(c, p, shares, base) || w.next(c, p));
            }
            for (uint32_t k = 0;; ++k) {
                Item *mine = &S.item[k % kItems];
                if (warp == kWalkWarp) {
                    if (k >= kItems && !wait(&S.item_empty[k % kItems], (k / kItems & 1) ^ 1))
                        break;
                    if (lane == 0) {
                        Item x{};
                        if (more) {
                            x.r = w.r;
                            x.h = w.first_head();
                            x.b = w.b;
                            x.rows = w.rows();
                            x.nt = w.t1 - w.t0;
                            x.t0 = w.t0;
                            x.tiles = w.tiles;
                            x.keys = w.range.keys;
                            x.near = w.range.near;
                            x.gap = w.range.gap;
                            x.kind = w.kind() + (MODE != kWhole && w.twins ? 4 : 0);
                            x.len = MODE == kShared && w.of_group ? w.q.tokens : w.q.len - w.range.gap;
                            x.n = MODE == kShared && w.of_group ? 0 : w.q.n;
                            x.first = p.cu[w.r];
                            x.q_use = q_use;
                            x.slots = slots;
                        }
                        *mine = x;
                        mbar_arrive(&S.item_full[k % kItems]);
                        if (more) {  // for the joins
                            if (w.t0 == 0 && w.t1 < w.tiles) {  // goes on behind the share
                                Partial &y = p.partial[blockIdx.x];
                                y.r = w.r;
                                y.h = w.h;
                                y.b = w.b;
                                y.rows = x.rows;
                                y.last_place = w.last;
                                y.shares = shares;
                            }
                            if (MODE == kShared && w.t0 == 0) {
                                const int m = w.b * kBlockRows, token = by_group(p, m);
                                const int64_t at = ((w.kind() == 1 ? 0 : p.N) + x.first + token) * p.heads +
                                                   x.h * p.group + m - token * p.group;
                                const int2 y = make_int2(blockIdx.x, w.t1 < w.tiles ? shares.owner(w.last) - (int)blockIdx.x + 1
                                                                                   : 0);
                                p.row_parts[at] = y;
                                if (w.twins)
                                    p.row_parts[at + p.group] = y;
                            }
                        }
                    }
                    __syncwarp();
                } else if (!announced(k)) {
                    break;
                }
                const Item item = *mine;
                if (warp != kWalkWarp)
                    done_with(k);
                if (item.nt == 0)
                    break;
                const bool twins = MODE != kWhole && item.kind & 4;
                const int count = item.rows > kTile || twins ? 2 : 1;
                q_use = item.q_use + count;
                slots = item.slots + (twins ? 4 : 2) * item.nt;
                constexpr int kVecs = DP / 8, kStep = 32 * kQueryWarps / kVecs;  // 16-byte units of a row, rows of a turn
                for (int g = 0; g < count; ++g) {
                    const int use = item.q_use + g;
                    if (use >= 2)
                        wait(&S.q_empty[use & 1], (use >> 1 & 1) ^ 1);
                    if (__any_sync(kFull, S.gave_up))
                        break;
                    arrivals += lane == (use & 1);
                    const int at = part * 32 + lane, vec = at % kVecs;
                    const uint32_t dst = smem_addr(qtile) + (use & 1) * Z::kSlotBytes + vec / 8 * Z::kChunk;
                    const int more_rows = twins ? 0 : g * kTile, h = item.h + (twins ? g : 0);
                    const int m0 = item.b * kBlockRows + more_rows, rows = min(kTile, item.rows - more_rows);
                    if (count == 2 && !twins && p.q_tokens) {
                        // a wide row block's: one copy for each 64 elements (rows behind the last are not
                        // looked at); row by row they took 7 us, with the products waiting
                        if (warp == kWalkWarp) {
                            if (elect_one()) {
                                mbar_arrive_expect_tx(&S.q_full[use & 1], Z::kSlotBytes);
#pragma unroll
                                for (int i = 0; i < DP / 64; ++i)
                                    tma_rows(smem_addr(qtile) + (use & 1) * Z::kSlotBytes + i * Z::kChunk, &qmap,
                                             i * 64, item.h * p.group, item.first + by_group(p, m0),
                                             &S.q_full[use & 1]);
                            }
                        } else if (lane == 0) {
                            mbar_arrive(&S.q_full[use & 1]);
                        }
                        __syncwarp();
                        continue;
                    }
                    int x = at / kVecs, token = by_group(p, m0 + x), head = (m0 + x) - token * p.group;
                    const int more_tokens = by_group(p, kStep), more_heads = kStep - more_tokens * p.group;
                    const char *src = p.q + 2 * ((int64_t)item.first * p.q_token +
                                                 (int64_t)(h * p.group) * p.q_head + vec * 8);
                    if (vec * 8 < c.dim) {
                        for (; x < rows; x += kStep) {
                            copy16(dst + x * 128 + ((vec % 8) ^ (x % 8)) * 16,
                                   src + 2 * (token * p.q_token + head * p.q_head));
                            token += more_tokens;
                            head += more_heads;
                            if (head >= p.group) {
                                head -= p.group;
                                ++token;
                            }
                        }
                    } else {
                        for (; x < rows; x += kStep)
                            zero16(dst + x * 128 + ((vec % 8) ^ (x % 8)) * 16);
                    }
                    asm volatile("cp.async.wait_all;" ::: "memory");
                    fence_proxy_async_shared();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&S.q_full[use & 1]);
                }
                if (warp == kWalkWarp)
                    more = w.next(c, p);
            }
            if (lane < 2)
                atomicAdd(&S.arrivals[SLOTS + lane], arrivals);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        const int g = warp >> 2, row = tid & (kTile - 1), sub = warp & 3;
        const uint32_t lanes = (uint32_t)sub * 32 << 16;
        const uint32_t s_addr = tmem + g * 256 + lanes;
        uint32_t s_turn = 0, o_turn = 0, merge_turn = 0;
        uint32_t wide_cuts = 0;
        int cuts = 0;  // row blocks so far with keys that some of their rows do not see
        // all eight softmax warps
        auto meet = [&]() {
            tmem_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&S.merge);
            wait(&S.merge, merge_turn);
            merge_turn ^= 1;
            tmem_fence_after();
        };
        // First one tile of nothing, while the first keys are on their way: it fetches the code (a first
        // tile took 5500 cycles, the others 2000), and ends before the first product writes S.
        bool dry = true;
        for (uint32_t k = 0;;) {
            Item item{};
            if (!dry) {
                if (!announced(k))
                    break;
                item = S.item[k % kItems];
                done_with(k);
                ++k;
            } else {
                item.rows = kTile;
                item.nt = 1 + g;
                item.keys = 4 * kTile;  // (and len 0: with masks)
            }
            const int nt = item.nt;
            if (nt == 0)
                break;
            // wide: both groups take every tile (twins: of a head each)
            const bool twins = MODE != kWhole && item.kind & 4, wide = item.rows > kTile || twins;
            const int m0 = wide && !twins ? g * kTile : 0;   // the group's first row in the block
            const int mine = min(kTile, item.rows - m0);     // its rows
            const bool warp_on = sub * 32 < mine, on = row < mine;
            const int m = item.b * kBlockRows + m0 + row;    // row of the request
            const int token = by_group(p, m), kv_head = item.h + (twins ? g : 0);
            const int q_head = kv_head * p.group + m - token * p.group;

            const int turns = wide ? nt : (nt - g + 1) / 2;  // this group's tiles

            uint32_t bits[kMaxTree / 32] = {};
            int depth = 0;  // windows: of the row's node
            bool refused = false;  // the request's tree is malformed: every row block of it is left out
            if (p.parent && !dry && !(MODE == kShared && (item.kind & 3) == 1)) {
                int32_t *par = S.group[g].parent;  // every warp of the group writes the same there
                bool bad = false;
                for (int i = lane; i < item.n; i += 32) {
                    const int up = p.parent[item.first + i];
                    bad |= i == 0 ? up != -1 : up < 0 || up >= i;
                    if (turns > 0)  // a group without tiles does not wait for its warps before it writes ml[] there
                        par[i] = up;
                }
                refused = __any_sync(kFull, bad);
                __syncwarp();
                if (refused) {
                    if (lane == 0)
                        cache_error(c.error, SPEC_DEVERR_TREE, item.r);
                } else if (on && turns > 0) {
                    // (ends whatever stands in par[]: the array may be written while other warps read it)
                    if (MODE == kWindow) {
                        for (int at = min(par[token], token - 1); at >= 0; at = min(par[at], at - 1))
                            ++depth;
                    }
                    int up = depth;  // the node's depth
                    for (int at = token; at >= 0; at = min(par[at], at - 1), --up) {
                        const bool seen = MODE != kWindow || up > depth - p.window || item.len + up < p.sinks;
#pragma unroll
                        for (int j = 0; j < kMaxTree / 32; ++j)
                            bits[j] |= at / 32 == j && seen ? 1u << (at & 31) : 0u;
                    }
                }
                __syncwarp();
            }
            const bool kept = on && !refused;  // the row has a result
            // keys that every row of this warp sees
            int all_see = p.parent ? item.len
                                   : item.len + by_group(p, item.b * kBlockRows + m0 + sub * 32) + 1;
            // ... and of the whole row block
            int common = p.parent ? item.len + (MODE != kWindow) : item.len + by_group(p, item.b * kBlockRows) + 1;
            // keys of the chain that this row sees end here
            int limit = item.len + token + 1;
            if (MODE == kShared && (item.kind & 3) == 1)
                all_see = common = limit = item.keys;
            const int last = min(item.keys, (item.t0 + nt) * kTile);
            // Windows: behind the sinks a row sees no key below `low`, at least up to its own; the highest of the row
            // block's is `high` or below it, of the warp's `warp_high`
            int low = 0, high = 0, warp_high = 0;
            if (MODE == kWindow) {
                const int most = p.parent ? item.n - 1 : by_group(p, item.b * kBlockRows + item.rows - 1);
                const int warp_most = by_group(p, item.b * kBlockRows + min(m0 + sub * 32 + 31, item.rows - 1));
                low = item.len + (p.parent ? depth : token) - p.window + 1;
                high = item.len + most - p.window + 1;
                warp_high = p.parent ? high : item.len + warp_most - p.window + 1;
                if (p.parent)
                    low = min(low, item.len);  // the tree's own keys go by `bits`
            }
            // keys of the share that lie below the window of some rows, or of all
            const int some_from = max(p.sinks, item.t0 * kTile), some = min(high, last);
            const bool cut_block = (last > common || (MODE == kWindow && some > some_from)) && !dry;
            cuts += cut_block;
            float M = -INFINITY, l = 0;
            bool any = false;  // the accumulator holds something
            for (int t = wide ? 0 : g; t < nt; t += wide ? 1 : 2) {
                if (!dry) {
                    wait(&S.s_full[g], s_turn);
                    s_turn ^= 1;
                }
                const int column = (item.t0 + t) * kTile;
                if (warp_on) {
                    tmem_fence_after();
                    // Keys that some row of the warp does not see: their scores become -inf where they lie, 32 at a
                    // time, so that neither look below has to ask.  (Asked in both: twice the work and four times the
                    // code; windows over prompts 104 us against 90, over trees 45 against 37, trees 53 against 48.)
                    if (column + kTile > all_see ||
                        (MODE == kWindow && column + kTile > p.sinks && column < warp_high)) {
#pragma unroll 1
                        for (int j = 0; j < kTile / 32; ++j) {
                            const int col = column + j * 32;
                            uint32_t see = p.parent ? tree_columns(bits, item.len, col) : low_bits(limit - col);
                            if (MODE == kWindow)
                                see &= low_bits(p.sinks - col) | ~low_bits(low - col);
                            if (__all_sync(kFull, see == ~0u))
                                continue;
                            float x[32];
                            tmem_ld32(s_addr + j * 32, x);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                x[e] = see >> e & 1 ? x[e] : -INFINITY;
                            tmem_st32(s_addr + j * 32, x);
                        }
                        tmem_wait_st();
                    }
                    // 64 columns at a time, read once for the maximum and once for the exponentials: the
                    // code of a tile is fetched anew by every block, and runs at a fetch's pace then
                    // (all 128 in registers, unrolled: 2% faster on prompt chunks, first tile 2 us)
                    auto columns = [&](int j, float *x) {
                        tmem_ld32(s_addr + j * 64, x);
                        tmem_ld32(s_addr + j * 64 + 32, x + 32);
                        tmem_wait_ld();
                    };
                    float mx = -INFINITY;
#pragma unroll 1
                    for (int j = 0; j < kTile / 64; ++j) {
                        float x[64];
                        columns(j, x);
                        float top[4] = {mx, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int e = 0; e < 64; e += 8)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                top[i] = max3(top[i], x[e + 2 * i], x[e + 2 * i + 1]);
                        mx = max3(fmaxf(top[0], top[1]), top[2], top[3]);
                    }
                    mx *= p.scale_log2;
                    // Also from -inf.  fp16, whose weights end at 2^16: of the difference, which is exact, as a sum
                    // may round up to twice the limit from 2^23 on.  (The exponents below are of products rounded
                    // once, with M taken off, so up to half a step of mx off: with the limit, which the difference
                    // then keeps by as much, 15.5 at most for products below 2^28.)  bf16 has the range for the
                    // sum (prompt chunks 326.2 us, 328.3 by the difference).
                    const bool grown = DT == SPEC_F16 ? mx - M > kHead<DT> + kLazy : mx > M + kLazy;
                    const float f = grown ? ex2(M - (mx - kHead<DT>)) : 1.0f;
                    if (grown) {
                        M = mx - kHead<DT>;
                        l *= f;
                    }
                    if (any && __any_sync(kFull, grown)) {
#pragma unroll 1
                        for (int j = 0; j < DP / 32; ++j) {
                            float o[32];
                            tmem_ld32(s_addr + kTile + j * 32, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                o[e] *= f;
                            tmem_st32(s_addr + kTile + j * 32, o);
                        }
                        tmem_wait_st();
                    }
                    any = true;
                    const float base = M == -INFINITY ? 0.0f : -M;
                    const uint64_t scale2 = pack2(p.scale_log2, p.scale_log2), base2 = pack2(base, base);
                    uint64_t sum[4] = {};
#pragma unroll 1
                    for (int j = 0; j < kTile / 64; ++j) {
                        float x[64];
                        columns(j, x);
#pragma unroll
                        for (int e = 0; e < 64; e += 2) {
                            float a, b;
                            unpack2(fma2(pack2(x[e], x[e + 1]), scale2, base2), a, b);
                            a = ex2(a);
                            b = ex2(b);
                            sum[e / 2 & 3] = add2(sum[e / 2 & 3], pack2(a, b));
                            // 16 bits, as the product with V takes them (the sum above does not lose them): errors
                            // against 64 bits of 0.0023 in bf16, where outputs alone rounded have 0.0017, and of
                            // 0.00027 beside 0.00021 in fp16
                            x[e / 2] = __uint_as_float(from_float2<DT>(a, b));
                        }
                        tmem_st32(s_addr + j * 32, x);
                    }
                    float a, b;
                    unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), a, b);
                    l += a + b;
                    tmem_wait_st();
                    tmem_fence_before();
                }
                // A weight of zero must meet a finite value: rows of V behind the last key become zeros,
                // whatever the page (or the slot before) holds there, and so do values that are not
                // finite at keys that only some of the rows see (add_spoilt() gives them to those).
                const int behind = item.keys - column, unseen = min(common - column, behind);
                // windows: keys from w0 to w1 are below the window of some rows or all
                const int w0 = MODE == kWindow ? min(max(p.sinks - column, 0), kTile) : 0,
                          w1 = MODE == kWindow ? max(min(min(high - column, kTile), unseen), 0) : 0;
                if ((unseen < kTile || (MODE == kWindow && w0 < w1)) && (!wide || g == 0 || twins) && !dry) {
                    const uint32_t use = item.slots + slot_of(true, twins, g, t, nt);
                    wait(&S.full[use % SLOTS], use / SLOTS & 1);
                    char *base = ring + use % SLOTS * Z::kSlotBytes;
                    const int i0 = max(unseen, 0) * 8 + row, i1 = min(behind, kTile) * 8;
                    auto look = [&](int i0, int i1) {
                        uint32_t bad = 0;
#pragma unroll 4
                        for (int i = i0; i < i1; i += kTile)
#pragma unroll
                            for (int j = 0; j < DP / 64; ++j) {
                                const uint4 x = *reinterpret_cast<const uint4 *>(base + j * Z::kChunk + i * 16);
                                bad |= not_finite<DT>(x.x) | not_finite<DT>(x.y) | not_finite<DT>(x.z) |
                                       not_finite<DT>(x.w);
                            }
                        if (bad & 0x80008000u) {
                            drop_not_finite<DT, DP>(base, i0, i1);
                            S.spoilt[twins ? g : 0][cuts & 1] = cuts;
                        }
                    };
                    look(i0, i1);
                    if (MODE == kWindow)
                        look(w0 * 8 + row, w1 * 8);
                    for (int i = i1 + row; i < kTile * 8; i += kTile)
#pragma unroll
                        for (int j = 0; j < DP / 64; ++j)
                            *reinterpret_cast<uint4 *>(base + j * Z::kChunk + i * 16) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_shared();
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(dry ? &S.ready : &S.p_full[g]);
            }
            if (dry) {
                dry = false;
                continue;
            }
            if (turns > 0) {
                wait(&S.o_full[g], o_turn);  // its last product
                o_turn ^= 1;
            }
            tmem_fence_after();
            const bool whole = item.t0 == 0 && nt == item.tiles;
            // partial sums: of a row block from before this share (0), or going on behind it (1)
            const int64_t place = ((int64_t)blockIdx.x * 2 + (item.t0 == 0)) * p.max_rows + m0 + row;
            char *out = p.out + 2 * ((int64_t)(item.first + token) * p.out_token + q_head * p.out_head);
            // of a row of a group: its place over the shared tokens, or over its own
            const int64_t in_group = (((item.kind & 3) - 1) * p.N + item.first + token) * p.heads + q_head;
            float *sums = MODE == kShared && whole ? p.row_o + in_group * DP : p.part_o + place * DP;
            const bool to_out = whole && (MODE != kShared || (item.kind & 3) == 0);
            auto store = [&](const float *o, int col, float by) {  // 32 columns
                if (!kept)
                    return;
                if (to_out) {
                    uint32_t y[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        y[e] = from_float2<DT>(o[2 * e] * by, o[2 * e + 1] * by);
#pragma unroll
                    for (int e = 0; e < 16; e += 8) {
                        if (p.out_by_32) {
                            if (col + 2 * e < c.dim)
                                store32(out + 2 * col + 4 * e, y + e);
                        } else {
#pragma unroll
                            for (int i = e; i < e + 8; i += 4)
                                if (col + 2 * i < c.dim)
                                    *reinterpret_cast<uint4 *>(out + 2 * col + 4 * i) =
                                        make_uint4(y[i], y[i + 1], y[i + 2], y[i + 3]);
                        }
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 32; e += 8)
                        store32(sums + col + e, reinterpret_cast<const uint32_t *>(o + e));
                }
            };
            auto store_ml = [&]() {
                if (!on)
                    return;
                if (!to_out)
                    *(MODE == kShared && whole ? p.row_ml + in_group : p.part_ml + place) =
                        refused ? make_float2(0, -1) : make_float2(M, l);
                else if (p.lse && kept)
                    p.lse[(int64_t)(item.first + token) * p.heads + q_head] = (M + log2f(l)) * 0.69314718055994531f;
            };
            // (The groups are less than two row blocks apart, by their meetings or, of wide ones, by the order
            // of the products: nobody writes spoilt[] for the next but one before all have read it here.)
            auto spoilt = [&]() {
                if (cut_block && kept && S.spoilt[twins ? g : 0][cuts & 1] == cuts) {
                    const uint4 tree = make_uint4(bits[0], bits[1], bits[2], bits[3]);
                    char *result = to_out ? out : reinterpret_cast<char *>(sums);
                    const int from = max(common, item.t0 * kTile);
                    add_spoilt<DT, MODE>(c, p, item.r, kv_head, from, last, item.near, item.gap, item.len, token, low, tree,
                                         result, !to_out);
                    if (MODE == kWindow)
                        add_spoilt<DT, MODE>(c, p, item.r, kv_head, some_from, min(some, from), item.near, item.gap, item.len,
                                             token, low, tree, result, !to_out);
                }
            };
            if (wide) {
                if (cut_block && !twins) {
                    if (g == 1)
                        wait(&S.known[wide_cuts & 1], wide_cuts >> 1 & 1);
                    else if (lane == 0)
                        mbar_arrive(&S.known[wide_cuts & 1]);
                    ++wide_cuts;
                }
                if (warp_on) {
#pragma unroll 1
                    for (int j = 0; j < DP / 32; ++j) {
                        float o[32];
                        tmem_ld32(s_addr + kTile + j * 32, o);
                        tmem_wait_ld();
                        store(o, j * 32, 1.0f / l);
                    }
                    store_ml();
                }
                spoilt();
            } else {
                S.group[g].ml[row] = make_float2(M, l);
                meet();
                if (warp_on) {
                    const float2 other = S.group[g ^ 1].ml[row];
                    const float top = fmaxf(M, other.x);
                    const float fm = M == -INFINITY ? 0.0f : ex2(M - top);
                    const float fo = other.x == -INFINITY ? 0.0f : ex2(other.x - top);
                    M = top;
                    l = l * fm + other.y * fo;
                    const float f0 = g == 0 ? fm : fo, f1 = g == 0 ? fo : fm;
                    const uint32_t o_addr = tmem + lanes + kTile + g * (DP / 2);  // half of the columns
#pragma unroll 1
                    for (int j = 0; j < DP / 64; ++j) {
                        float o[32];
                        tmem_ld32(o_addr + j * 32, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] *= f0;
                        if (nt > 1) {
                            float o1[32];
                            tmem_ld32(o_addr + 256 + j * 32, o1);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                o[e] = fmaf(o1[e], f1, o[e]);
                        }
                        store(o, g * (DP / 2) + j * 32, 1.0f / l);
                    }
                    if (g == 0)
                        store_ml();
                }
                meet();
                if (g == 0)  // (both halves are written; the other group may have had no tile, and no bits)
                    spoilt();
            }
        }
        tmem_fence_before();
    }
    __syncthreads();
    if (warp == 10 && S.gave_up && lane < SLOTS + 2) {
        // copies that nobody waited for: a lane per barrier
        uint64_t *bar = lane < SLOTS ? &S.full[lane] : &S.q_full[lane - SLOTS];
        const Drain d = drain_of(S.arrivals[lane], lane < SLOTS ? 2 : kQueryWarps);
        for (uint32_t i = 0; i < d.missing; ++i)
            mbar_arrive(bar);
        for (uint32_t i = 0; d.begun && i < kWaitLimit && !mbar_try_wait(bar, d.parity); ++i) {
        }
    }
    __syncthreads();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == kMmaWarp) {
        tmem_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemColumns));
    }
}

// Joins the partial sums of the row blocks that were cut: blocks (share, y), W warps per row, each for
// every W-th part, J rows per warp at the same time.  Bound by the latency of L2, a chain of three loads
// (the row block, the weights, the parts): two parts of every row are on their way before the weights
// are known.
template <int DT, int DP, int W, int J>
__device__ __forceinline__ void join(const CacheView &c, const AttentionParams &p, const Partial &x, float4 (*sums)[32],
                                     int row0, int lane, int warp)
{
    const int mine = warp % W, next = gridDim.y * (8 / W);  // from a row of the warp's to its next
    const int parts = x.shares.owner(x.last_place) - (int)blockIdx.x + 1;
    // the first part is the tail of its block's share, the others lie at the head of theirs; rows behind
    // the last are the first over again
    auto place = [&](int i, int j) {
        const int row = row0 + j * next;
        return part_place(blockIdx.x, i, p.max_rows, row < x.rows ? row : row0);
    };
    constexpr int E = DP / 32;  // elements per lane
    auto load = [&](int i, int j, float *v) {
        const float *o = p.part_o + place(i, j) * DP + lane * E;
        if (E == 4) {
            const float4 y = *reinterpret_cast<const float4 *>(o);
            v[0] = y.x, v[1] = y.y, v[2] = y.z, v[3] = y.w;
        } else {
            const float2 y = *reinterpret_cast<const float2 *>(o);
            v[0] = y.x, v[1] = y.y;
        }
    };
    float top[J], l[J], acc[J][4];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        top[j] = -INFINITY;
        l[j] = 0;
        acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0;
    }
    // 32 parts in a turn, nearly always all
#pragma unroll 1
    for (int i0 = 0; i0 < parts; i0 += 32) {
        const int some = min(32, parts - i0);
        float2 ml[J];
        // two parts on their way before the weights are known
        const int a = mine, b = mine + W;
        float va[J][4], vb[J][4];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            ml[j] = lane < some ? p.part_ml[place(i0 + lane, j)] : make_float2(-INFINITY, 0);
            load(i0 + min(a, some - 1), j, va[j]);
            load(i0 + min(b, some - 1), j, vb[j]);
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const float now = fmaxf(top[j], warp_max(ml[j].x)), f = top[j] == -INFINITY ? 0.0f : ex2(top[j] - now);
            top[j] = now;
            ml[j].x = ml[j].x == -INFINITY ? 0.0f : ex2(ml[j].x - now);
            l[j] = l[j] * f + warp_sum(ml[j].x * ml[j].y);
            const float fa = __shfl_sync(kFull, ml[j].x, a), fb = __shfl_sync(kFull, ml[j].x, b);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (i0 > 0)
                    acc[j][e] *= f;
                if (a < some)
                    acc[j][e] = fmaf(fa, va[j][e], acc[j][e]);
                if (b < some)
                    acc[j][e] = fmaf(fb, vb[j][e], acc[j][e]);
            }
        }
#pragma unroll(8 / J)
        for (int i = mine + 2 * W; i < some; i += W) {
#pragma unroll
            for (int j = 0; j < J; ++j) {
                float v[4];
                load(i0 + i, j, v);
                const float f = __shfl_sync(kFull, ml[j].x, i);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    acc[j][e] = fmaf(f, v[e], acc[j][e]);
            }
        }
    }
    if (W > 1) {
        sums[warp][lane] = make_float4(acc[0][0], acc[0][1], acc[0][2], acc[0][3]);
        asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / W), "n"(32 * W) : "memory");
        if (mine > 0)
            return;
#pragma unroll
        for (int i = 1; i < W; ++i) {
            const float4 y = sums[warp + i][lane];
            acc[0][0] += y.x, acc[0][1] += y.y, acc[0][2] += y.z, acc[0][3] += y.w;
        }
    }
    const int first = p.cu[x.r];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int row = row0 + j * next;
        if (row >= x.rows)
            return;
        if (l[j] < 0)
            continue;  // of a refused request: its parts have sums of -1
        const int m = x.b * kBlockRows + row;
        const int token = by_group(p, m), head = x.h * p.group + m - token * p.group;
        const int64_t t = (int64_t)first + token;
        const float by = 1.0f / l[j];
        if (lane * E < c.dim) {
            char *out = p.out + 2 * (t * p.out_token + head * p.out_head + lane * E);
            const uint32_t low = from_float2<DT>(acc[j][0] * by, acc[j][1] * by);
            if (E == 4)
                *reinterpret_cast<uint2 *>(out) = make_uint2(low, from_float2<DT>(acc[j][2] * by, acc[j][3] * by));
            else
                *reinterpret_cast<uint32_t *>(out) = low;
        }
        if (lane == 0 && p.lse)
            p.lse[t * p.heads + head] = (top[j] + log2f(l[j])) * 0.69314718055994531f;
    }
}

// Row blocks of many rows are cut into few parts (a warp for up to kJoinRows rows; prompt chunks with 1, 2
// and 4 rows per warp: 314, 312 and 316 us), those of few rows into as many as there are SMs (four warps per
// row: 38 parts of 48 rows took 79 us in all with one, 62 with four).
constexpr int kJoinRows = 2;

template <int DT, int DP, int W>
__global__ void __launch_bounds__(256) join_kernel(CacheView c, AttentionParams p)
{
    __shared__ float4 sums[W > 1 ? 8 : 1][32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row0 = blockIdx.y * (8 / W) + warp / W;
    const Partial x = p.partial[blockIdx.x];
    if (row0 >= x.rows)
        return;
    if (W > 1 || row0 + gridDim.y * 8 >= x.rows)
        join<DT, DP, W, 1>(c, p, x, sums, row0, lane, warp);
    else
        join<DT, DP, W, kJoinRows>(c, p, x, sums, row0, lane, warp);
}

// Joins what the rows of a call with shared prefixes have from their group's tokens and from their own, each in one
// piece or in the parts that it was cut into.  Blocks (request, y), a warp per row, of requests of about as many rows up
// to kJoinShared of them in turn.  Bound by latency, a chain of three loads (the request, its row blocks, their sums).
// The blocks per request are those of an average one's rows, so a step in which one request has most of the rows keeps
// few warps busy: 127 requests of one token and one of 2048, 32/8 heads of 128, behind 2048 shared tokens 882 us, without
// sharing 340; where no request is in a group, 490 and 345.
constexpr int kJoinShared = 4;  // (2 / 4 / 8: a verify step of 1152 tokens 235 / 234.5 / 238 us in all)

template <int DT, int DP> __global__ void __launch_bounds__(256) join_shared_kernel(CacheView c, AttentionParams p)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 q = p.requests[blockIdx.x];
    const int begun = *p.begun, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (!begun || q.x == 0)
        return;
    constexpr int E = DP / 32, U = 4;  // elements per lane, parts on their way before the weights are known
    const int rows = q.x * c.heads;    // head by head, so that a warp's next row has mostly the same row blocks
#pragma unroll 1
    for (int i = blockIdx.y * 8 + warp; i < rows; i += gridDim.y * 8) {
        const int kv = (uint32_t)i / (uint32_t)q.x, m = i - kv * q.x, token = by_group(p, m);
        const int head = kv * p.group + m - token * p.group;
        const int64_t t = (int64_t)q.y + token, at = t * p.heads + head;
        // a row's place in the row blocks of the group and of the request, and what became of them
        auto parts_of = [&](int m, int from, int64_t side, int *row) {
            const int first = m & -kBlockRows, token = by_group(p, first);
            *row = m - first;
            return p.row_parts[(side + from + token) * p.heads + kv * p.group + first - token * p.group];
        };
        int row_a = 0, row_b;
        const int2 b = parts_of(m, q.y, p.N, &row_b);
        int2 a = make_int2(0, 0);
        if (q.z)
            a = parts_of(m + (q.y - q.w) * p.group, q.w, 0, &row_a);
        else if (b.y == 0)
            continue;  // nothing to join: it is in out
        if (!parts_within(a.x, a.y, p.blocks) || !parts_within(b.x, b.y, p.blocks))
            continue;  // never written: a wait gave up
        const int in_a = q.z ? max(a.y, 1) : 0, parts = in_a + max(b.y, 1);
        // where part k's sums are: its place among those of cut row blocks, or below zero the row's
        auto place = [&](int k) {
            const bool own = k >= in_a;
            const int2 x = own ? b : a;
            const int j = own ? k - in_a : k;
            return x.y > 0 ? part_place(x.x, j, p.max_rows, own ? row_b : row_a)
                           : -1 - (at + (own ? p.N * p.heads : 0));
        };
        auto load = [&](int k, float *v) {
            const int64_t x = place(k);
            const float *o = (x >= 0 ? p.part_o + x * DP : p.row_o + (-1 - x) * DP) + lane * E;
            if (E == 4) {
                const float4 y = *reinterpret_cast<const float4 *>(o);
                v[0] = y.x, v[1] = y.y, v[2] = y.z, v[3] = y.w;
            } else {
                const float2 y = *reinterpret_cast<const float2 *>(o);
                v[0] = y.x, v[1] = y.y;
            }
        };
        float top = -INFINITY, l = 0, acc[4] = {};
        bool refused = false;
#pragma unroll 1
        for (int k0 = 0; k0 < parts; k0 += 32) {
            const int some = min(32, parts - k0);
            float2 ml = make_float2(-INFINITY, 0);
            if (lane < some) {
                const int64_t x = place(k0 + lane);
                ml = x >= 0 ? p.part_ml[x] : p.row_ml[-1 - x];
            }
            float v[U][4];
#pragma unroll
            for (int u = 0; u < U; ++u)
                load(k0 + min(u, some - 1), v[u]);
            refused |= __any_sync(kFull, ml.y < 0);
            const float now = fmaxf(top, warp_max(ml.x)), f = top == -INFINITY ? 0.0f : ex2(top - now);
            top = now;
            const float w = ml.x == -INFINITY ? 0.0f : ex2(ml.x - now);
            l = l * f + warp_sum(w * ml.y);
            if (k0 > 0)
#pragma unroll
                for (int e = 0; e < E; ++e)
                    acc[e] *= f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float x = __shfl_sync(kFull, w, u);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (u < some)
                        acc[e] = fmaf(x, v[u][e], acc[e]);
            }
#pragma unroll 4
            for (int k = U; k < some; ++k) {
                load(k0 + k, v[0]);
                const float x = __shfl_sync(kFull, w, k);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    acc[e] = fmaf(x, v[0][e], acc[e]);
            }
        }
        if (refused)
            continue;  // its parts have sums of -1
        const float by = 1.0f / l;
        if (lane * E < c.dim) {
            char *out = p.out + 2 * (t * p.out_token + head * p.out_head + lane * E);
            const uint32_t low = from_float2<DT>(acc[0] * by, acc[1] * by);
            if (E == 4)
                *reinterpret_cast<uint2 *>(out) = make_uint2(low, from_float2<DT>(acc[2] * by, acc[3] * by));
            else
                *reinterpret_cast<uint32_t *>(out) = low;
        }
        if (lane == 0 && p.lse)
            p.lse[at] = (top + log2f(l)) * 0.69314718055994531f;
    }
}

// ---------------------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------------------

struct AttentionPlan {
    int dp, max_rows;
    size_t partial, ml, o, begun, requests, row_parts, row_ml, row_o, total;
};

AttentionPlan attention_plan(const CacheView &c, int32_t num_q_heads, int64_t N, bool shared)
{
    AttentionPlan a;
    a.dp = c.dim <= 64 ? 64 : 128;
    a.max_rows = (int)std::max<int64_t>(1, std::min<int64_t>(kBlockRows, N * (num_q_heads / c.heads)));
    size_t o = 0;
    a.partial = o;
    o = align256(o + sizeof(Partial) * kMaxGrid);
    a.ml = o;
    o = align256(o + sizeof(float2) * 2 * kMaxGrid * a.max_rows);
    a.o = o;
    o = align256(o + sizeof(float) * 2 * kMaxGrid * a.max_rows * a.dp);
    const int64_t rows = shared ? 2 * N * num_q_heads : 0;
    a.begun = o;
    o = align256(o + (shared ? sizeof(int32_t) : 0));
    a.requests = o;
    o = align256(o + (shared ? sizeof(int4) * (size_t)c.num_requests : 0));
    a.row_parts = o;
    o = align256(o + sizeof(int2) * rows);
    a.row_ml = o;
    o = align256(o + sizeof(float2) * rows);
    a.row_o = o;
    o = align256(o + sizeof(float) * rows * a.dp);
    a.total = o + 256;  // slack for aligning the caller's pointer
    return a;
}

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled()
{
    static const EncodeTiled f = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return f;
}

// The pages of one layer as a tensor (head_dim, token, head, page); a copy brings 64 elements of `box`
// tokens to shared memory, with the 128-byte swizzle that the products read.  What lies behind
// head_dim reads as zeros.  (One copy for both 64-element halves of a row, through a tensor of five
// dimensions, halves the copies and was slower: 180 ns per 4 KB copy against 43 ns per 2 KB.)
bool encode_pages(CUtensorMap *map, const CacheView &c, int dtype, char *base, int box)
{
    const EncodeTiled f = encode_tiled();
    if (!f)
        return false;
    const cuuint64_t least = 2 * (cuuint64_t)c.dim;  // any valid stride does for a dimension of size 1
    const cuuint64_t dims[4] = {(cuuint64_t)c.dim, (cuuint64_t)c.page_size, (cuuint64_t)c.heads,
                                (cuuint64_t)c.num_pages};
    const cuuint64_t strides[3] = {c.page_size > 1 ? 2 * (cuuint64_t)c.token_stride : least,
                                   c.heads > 1 ? 2 * (cuuint64_t)c.head_stride : least,
                                   c.num_pages > 1 ? 2 * (cuuint64_t)c.page_stride : least};
    const cuuint32_t boxes[4] = {64, (cuuint32_t)box, 1, 1}, steps[4] = {1, 1, 1, 1};
    return f(map, dtype == SPEC_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, base,
             dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The queries as a tensor (head_dim, head, token), whose boxes are the 128 rows of a softmax group.
bool encode_queries(CUtensorMap *map, const CacheView &c, int dtype, const AttentionParams &p)
{
    const EncodeTiled f = encode_tiled();
    if (!f)
        return false;
    const cuuint64_t least = 2 * (cuuint64_t)c.dim;
    const cuuint64_t dims[3] = {(cuuint64_t)c.dim, (cuuint64_t)p.heads, (cuuint64_t)p.N};
    const cuuint64_t strides[2] = {p.heads > 1 ? 2 * (cuuint64_t)p.q_head : least,
                                   p.N > 1 ? 2 * (cuuint64_t)p.q_token : least};
    const cuuint32_t boxes[3] = {64, (cuuint32_t)p.group, (cuuint32_t)p.q_tokens}, steps[3] = {1, 1, 1};
    return f(map, dtype == SPEC_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
             const_cast<char *>(p.q), dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DT, int DP, int MODE> cudaError_t prepare_kernel()
{
    return cudaFuncSetAttribute(attention_kernel<DT, DP, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                AttnSizes<DP>::kBytes);
}

// SMs of the current device; sets the kernels' shared memory on its first call there.
template <int MODE> cudaError_t prepare_kernels(int *sms)
{
    static int cached[kMaxDevices];  // written with the same value by every thread that finds it 0
    int dev;
    cudaError_t e = cudaGetDevice(&dev);
    if (e)
        return e;
    if (dev < 0 || dev >= kMaxDevices)
        return cudaErrorInvalidDevice;
    int n = __atomic_load_n(&cached[dev], __ATOMIC_ACQUIRE);
    if (n == 0) {
        e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (!e)
            e = prepare_kernel<SPEC_BF16, 64, MODE>();
        if (!e)
            e = prepare_kernel<SPEC_BF16, 128, MODE>();
        if (!e)
            e = prepare_kernel<SPEC_F16, 64, MODE>();
        if (!e)
            e = prepare_kernel<SPEC_F16, 128, MODE>();
        if (e)
            return e;
        __atomic_store_n(&cached[dev], n, __ATOMIC_RELEASE);
    }
    *sms = n;
    return cudaSuccess;
}

template <int DT, int DP, int MODE>
cudaError_t launch_attention(const CUtensorMap &kmap, const CUtensorMap &vmap, const CUtensorMap &qmap,
                             const CacheView &c, const AttentionParams &p, cudaStream_t st)
{
    const int grid = p.blocks;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 0;  // what other calls launched before, some as dependents of one another, has all ended
    cfg.stream = st;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kAttnThreads);
    cfg.dynamicSmemBytes = AttnSizes<DP>::kBytes;
    cudaError_t e = cudaLaunchKernelEx(&cfg, attention_kernel<DT, DP, MODE>, kmap, vmap, qmap, c, p);
    if (e)
        return e;
    cfg.numAttrs = 1;  // the join starts as the blocks end, and waits for the last of them itself
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    if constexpr (MODE == kShared) {
        const int64_t all = p.N * p.heads, rows = (all + p.B - 1) / p.B;  // of a request, on average
        const int64_t turns = std::max<int64_t>(1, std::min<int64_t>(kJoinShared, all / (grid * 40)));  // of a warp
        cfg.gridDim = dim3(p.B, (unsigned)std::min<int64_t>((rows + 8 * turns - 1) / (8 * turns), 65535));
        return cudaLaunchKernelEx(&cfg, join_shared_kernel<DT, DP>, c, p);
    } else {
        const int warps = p.max_rows <= 64 ? 4 : 1;  // per row
        const int rows = warps == 4 ? 2 : 8 * kJoinRows;  // per block
        cfg.gridDim = dim3(grid, (p.max_rows + rows - 1) / rows);
        return warps == 4 ? cudaLaunchKernelEx(&cfg, join_kernel<DT, DP, 4>, c, p)
                          : cudaLaunchKernelEx(&cfg, join_kernel<DT, DP, 1>, c, p);
    }
}

spec_status check_attention(const spec_cache *cache, CacheView *c, int32_t num_q_heads, int32_t B, int64_t N)
{
    spec_status s = view_cache(cache, c);
    if (s != SPEC_OK)
        return s;
    if (B < 0 || B > c->num_requests || N < 0 || num_q_heads < 1 || num_q_heads % c->heads)
        return SPEC_ERR_INVALID_ARG;
    if (c->dim > SPEC_ATTENTION_MAX_HEAD_DIM || c->page_size % 8 || num_q_heads / c->heads > 128 ||
        N * num_q_heads > INT32_MAX / 2)
        return SPEC_ERR_UNSUPPORTED;
    return SPEC_OK;
}

// What the entry points take.
struct AttentionCall {
    int32_t layer;
    const void *q;
    int64_t q_token_stride, q_head_stride;
    int32_t num_q_heads;
    const int32_t *cu_new;
    int32_t B;
    int64_t N;
    const int32_t *parent;
    float scale;
    void *out;
    int64_t out_token_stride, out_head_stride;
    float *lse;
    void *workspace;
    size_t workspace_bytes;
    void *stream;
    int32_t window, sinks;
    const int32_t *shared;
};

// The checks and launches of an entry point.
template <int MODE> spec_status attend(const spec_cache *cache, const AttentionCall &a)
{
    CacheView c;
    spec_status s = check_attention(cache, &c, a.num_q_heads, a.B, a.N);
    if (s != SPEC_OK)
        return s;
    if (a.layer < 0 || a.layer >= c.num_layers || !a.cu_new || !ptr_aligned(a.cu_new, 4) || !ptr_aligned(a.parent, 4) ||
        (a.N > 0 && (!a.q || !a.out)) || !ptr_aligned(a.q, 16) || !ptr_aligned(a.out, 16) || !ptr_aligned(a.lse, 4) ||
        !a.workspace || !(a.scale > 0) || !(a.scale < INFINITY))
        return SPEC_ERR_INVALID_ARG;
    if (!good_stride(a.q_token_stride, a.N) || !good_stride(a.out_token_stride, a.N) ||
        !good_stride(a.q_head_stride, a.num_q_heads) || !good_stride(a.out_head_stride, a.num_q_heads))
        return SPEC_ERR_INVALID_ARG;
    if ((MODE == kWindow && (a.window < 1 || a.sinks < 0)) ||
        (MODE == kShared && ((a.B > 0 && !a.shared) || !ptr_aligned(a.shared, 16))))
        return SPEC_ERR_INVALID_ARG;
    const AttentionPlan plan = attention_plan(c, a.num_q_heads, a.N, MODE == kShared);
    if (a.workspace_bytes < plan.total)
        return SPEC_ERR_WORKSPACE;
    int sms;
    if (cudaPeekAtLastError() != cudaSuccess || prepare_kernels<MODE>(&sms) != cudaSuccess)
        return SPEC_ERR_CUDA;
    if (a.B == 0 || a.N == 0)
        return SPEC_OK;
    AttentionParams p{};
    p.q = static_cast<const char *>(a.q);
    p.v = c.v + 2 * a.layer * c.layer_stride;
    p.out = static_cast<char *>(a.out);
    p.lse = a.lse;
    p.q_token = a.N > 1 ? a.q_token_stride : 0;
    p.out_token = a.N > 1 ? a.out_token_stride : 0;
    p.q_head = a.num_q_heads > 1 ? a.q_head_stride : 0;
    p.out_head = a.num_q_heads > 1 ? a.out_head_stride : 0;
    p.heads = a.num_q_heads;
    p.group = a.num_q_heads / c.heads;
    // 1 / group in 31 + ceil(log2(group)) bits, rounded up: it is off by less than group / 2^bits <=
    // 2^-31, too little to move the floor of m / group for any m < 2^31
    p.group_shift = 31;
    while ((1 << (p.group_shift - 31)) < p.group)
        ++p.group_shift;
    p.group_mul = (uint32_t)((((uint64_t)1 << p.group_shift) + p.group - 1) / p.group);
    p.B = a.B;
    p.blocks = std::min(sms, kMaxGrid);
    p.N = a.N;
    p.cu = a.cu_new;
    p.parent = a.parent;
    p.scale_log2 = a.scale * kLog2e;
    p.out_by_32 = ptr_aligned(a.out, 32) && p.out_token % 16 == 0 && p.out_head % 16 == 0 && c.dim % 16 == 0;
    char *ws = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(a.workspace) + 255) & ~uintptr_t(255));
    p.partial = reinterpret_cast<Partial *>(ws + plan.partial);
    p.part_ml = reinterpret_cast<float2 *>(ws + plan.ml);
    p.part_o = reinterpret_cast<float *>(ws + plan.o);
    p.max_rows = plan.max_rows;
    p.window = std::min(a.window, INT32_MAX / 2);  // more than there are positions: they and these add up in 32 bits
    p.sinks = std::min(a.sinks, INT32_MAX / 2);
    p.shared = reinterpret_cast<const int4 *>(a.shared);
    p.begun = reinterpret_cast<int32_t *>(ws + plan.begun);
    p.requests = reinterpret_cast<int4 *>(ws + plan.requests);
    p.row_parts = reinterpret_cast<int2 *>(ws + plan.row_parts);
    p.row_ml = reinterpret_cast<float2 *>(ws + plan.row_ml);
    p.row_o = reinterpret_cast<float *>(ws + plan.row_o);
    // (only where a row block can have more than 128 rows)
    p.q_tokens = kTile % p.group == 0 && a.N * p.group > kTile ? kTile / p.group : 0;
    p.box = 8;
    while (p.box < kTile && c.page_size % (2 * p.box) == 0)
        p.box *= 2;
    CUtensorMap kmap, vmap, qmap{};
    if (!encode_pages(&kmap, c, cache->dtype, c.k + 2 * a.layer * c.layer_stride, p.box) ||
        !encode_pages(&vmap, c, cache->dtype, c.v + 2 * a.layer * c.layer_stride, p.box) ||
        (p.q_tokens && !encode_queries(&qmap, c, cache->dtype, p)))
        return SPEC_ERR_UNSUPPORTED;
    cudaStream_t st = static_cast<cudaStream_t>(a.stream);
    cudaError_t e;
    if (cache->dtype == SPEC_BF16)
        e = plan.dp == 64 ? launch_attention<SPEC_BF16, 64, MODE>(kmap, vmap, qmap, c, p, st)
                          : launch_attention<SPEC_BF16, 128, MODE>(kmap, vmap, qmap, c, p, st);
    else
        e = plan.dp == 64 ? launch_attention<SPEC_F16, 64, MODE>(kmap, vmap, qmap, c, p, st)
                          : launch_attention<SPEC_F16, 128, MODE>(kmap, vmap, qmap, c, p, st);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // namespace
}  // namespace specrej

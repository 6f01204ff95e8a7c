// Kernel-level interfaces of the stacked-block operators: Newton-Schulz orthogonalisation of
// stacks of equal blocks and its gradient, the Muon step on them, global norm and AdamW.
//
// Every launch takes its descriptors by value as kernel parameters (up to 32 KB), so a call
// uploads nothing, keeps nothing between calls and can be captured as it stands.
#pragma once
#include <cuda.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "kernels.cuh"

namespace muon {

// ------------------------------------------------------------------ chains of fp16 products
// One launch runs a whole chain: a list of operations, each a product for every block of a class
//   out[b] = f_b * (alpha * sum_seg A_seg[b] x B_seg[b] + beta * (E0[b] + E1[b])) - diag * I,
// f_b = info[b][0]^pow, fp16 operands with fp32 accumulation in TMEM.  An operation of a block starts when
// the block's operations before it are done; blocks do not wait for each other.
//
// A class's planes lie in slots (iterations, or ping and pong) of `count` dense matrices one behind the
// other; a tensor map covers all slots of a plane.
constexpr uint32_t kStackAMn = 1u;       // A is contiguous along M (else along K)
constexpr uint32_t kStackBMn = 2u;       // B is contiguous along N (else along K)
constexpr uint32_t kStackSym = 4u;       // symmetric output: upper tiles computed, stored mirrored
constexpr uint32_t kStackOutBf16 = 8u;   // plane 0 of the output is bf16
constexpr uint32_t kStackRowMajor = 16u; // tiles swept along the rows of a block first
constexpr uint32_t kStackRescale = 32u;  // alpha and beta are multiplied by a power of two of the block's own (GradScale)

enum StackPlane { kPlaneX, kPlaneL, kPlaneA, kPlaneB, kPlaneOut, kPlaneD, kPlaneDL, kPlaneS, kPlaneP, kPlanes, kPlaneNone = 255 };
enum StackMap { kMapX, kMapA, kMapB, kMapD, kMapS, kMapP, kMaps };

// How the planes of a block's gradient D_t are scaled in the reverse pass: they hold D_t * 2^(k + e), and `sum` is the sum
// of the squares of what they hold, in units of 2^-30.  One per iterate, t = 0 .. iterations.
struct GradScale {
    unsigned long long sum;
    int e, unused;
};

struct ChainPlane {
    __half* p;
    long long block;       // elements between blocks
    int ld;                // elements between rows
};
struct alignas(64) ChainClass {
    CUtensorMap map[kMaps];
    ChainPlane plane[kPlanes];
    const float* info;     // kStackInfo floats per block
    int* done;             // per block: epilogue warps that have finished a tile
    int rp, cp, r8;        // padded sides of a block, padded shorter side
    int rows;              // rows that kPlaneOut takes
    int count;
    int scales;            // GradScales of a block
    GradScale* scale;      // kStackRescale: of the first block
};
struct ChainOp {
    float alpha, beta, diag;
    float room;            // kStackRescale: what the norm of the planes read may be multiplied up to
    int tile0;             // first tile of the operation in the launch (filled by the launcher)
    int need;              // value of `done` at which a block's operation may start (filled by the caller)
    uint8_t cls, kind;     // kind 0: r8 x r8 over the long side, 1: r8 x r8 over r8, 2: rp x cp over r8
    uint8_t flags, nseg, pow;
    uint8_t bn;            // tile width / 64: 1, 2 or 4
    uint8_t ma[2], mb[2];  // tensor maps of the segments' operands
    uint8_t sa[2], sb[2];  // and their slots
    uint8_t e[2], es[2];   // planes and slots of E
    uint8_t o[2], os[2];   // and of the output
    uint8_t t;             // kStackRescale: the iterate that is written; t + 1 is read
};
constexpr int kChainWarps = 16;          // epilogue warps of a tile: what a finished tile adds to `done`
constexpr int kChainMaxClasses = 12, kChainMaxOps = 360;

// Tensor map of `count` row-major fp16 matrices (rows x cols, dense): boxes of 64 x 64 of one matrix, 128-byte
// swizzle, zero fill out of bounds.  The same box serves as a K-major and as an MN-major piece of an operand.
bool encode_stack_tmap(CUtensorMap* out, const void* base, int rows, int cols, int count);

// Tiles of one block of an operation: 256 rows x 64 bn columns.  Symmetric ones are those that reach the upper
// triangle: with 4 / bn tile columns to 256, column nb has nb / (4 / bn) + 1 of them.
__host__ __device__ inline int chain_tiles(const ChainClass& c, const ChainOp& o) {
    const int w = 64 * o.bn, per = 4 / o.bn;
    if (o.kind == 2) return ((c.rp + 255) / 256) * ((c.cp + w - 1) / w);
    const int nbs = (c.r8 + w - 1) / w, whole = nbs / per, rest = nbs - whole * per;
    return per * whole * (whole + 1) / 2 + rest * (whole + 1);
}
// Launches ops[0 .. n) (in order; dependencies point backwards).  `ticket`: an int of the workspace that
// is zero; `done` counters carry on from earlier launches of the chain.
cudaError_t stack_chain_launch(const ChainClass* classes, int nc, ChainOp* ops, int n, int* ticket, unsigned* d_status,
                               int num_sms, cudaStream_t stream);

// ------------------------------------------------------------------ elementwise passes
// A run of blocks of one stack, as the elementwise kernels see it.  Element (b, i, j) of a
// caller's array is p[b * stride + i * ld + j]; of a workspace plane, q[b * rp * cp + i * cp + j]
// with rows and columns padded to multiples of 8 (zero there).
struct alignas(16) StackItem {
    const void* G;        // input or gradient
    float* M;             // momentum (nullable)
    void* W;              // weights or output
    __half* hi;           // workspace planes of the first block
    __half* lo;
    const __half* hi2;    // gradient of the input only: X_0
    float* info;          // per block: kStackInfo floats
    const float* ginfo;   // gradient of the input only: info of the gradient planes
    double* partials;     // per block: `chunks` doubles
    long long g_stride, m_stride, w_stride;
    int g_ld, m_ld, w_ld;
    int rows, cols, count;
    int chunks, per;      // chunks of per * kStackGroup padded elements in a block
    int chunk0;           // first chunk of this item in the launch
    int g_dtype, w_dtype;
    int vec;              // bit 0: G, bit 1: M, bit 2: W allow 8-element vector accesses
    float decay, step;    // W <- decay * W + step * X (step kernels); X * step (output, kPackGrad: a power of two)
    int* done;            // kPack, kPackGrad: per block, set to zero
    GradScale* scale;     // kPackGrad: per block, set to the planes' scale (last) and to zero; kGradOut: the first is D_0's
};
constexpr int kStackMaxItems = 128;
constexpr int kStackThreads = 256;
constexpr int kStackGroup = 8 * kStackThreads;
// (148 SMs, as the architecture has: a size query, which may run without a device, and the call must come to the same.)
// Groups of a CTA: one where that spreads few elements over more SMs (a pass over 2 x 320 x 257 took 13 us with
// four), four where there is work for all (24 x 512 x 1024: 41 us for the passes, 57 with one), and where a
// block's CTAs would add up too many partial sums.
inline int stack_per(int rp, int cp, int count) {
    return static_cast<long long>(rp) * cp * count > 148ll * 8 * kStackGroup ? 4 : 1;
}
inline int stack_chunks(int rp, int cp, int per) {
    const long long chunk = static_cast<long long>(per) * kStackGroup;
    return static_cast<int>((static_cast<long long>(rp) * cp + chunk - 1) / chunk);
}
// Per block: info[0] = f0 (X_0 = f0 * hi), info[1] = 2^k (hi = U * 2^k), info[2] = 1 / (N + eps),
// info[3] = N
constexpr int kStackInfo = 4;
constexpr int kStackTickets = 64;

enum class StackPass {
    kNorm,      // partials <- sum of U^2 (M updated in place where there is one)
    kPack,      // info <- norms; hi, lo <- U * 2^k
    kPackGrad,  // info2, scale <- norms; hi, lo <- G * 2^k * step (G: gradient of the output)
    kOut,       // W <- hi * step
    kUpdate,    // W <- decay * W + step * hi
    kDot,       // partials <- sum of (hi + lo) * hi2
    kGradOut,   // W <- gradient of the input
};
struct StackPassArgs {
    float beta;             // momentum coefficient
    int nesterov;
    float eps;
    const float* gscale;    // device: factor of G (nullable: 1)
    int* tickets;           // kPack, kPackGrad: kStackTickets ints set to zero
    int iters;              // kPackGrad, kGradOut
    unsigned* status;       // kNorm: cleared (unless null); kPack, kPackGrad: told of a norm that is not finite
};
cudaError_t stack_pass_launch(StackPass pass, StackItem* items, int n, const StackPassArgs& args, cudaStream_t stream);

// ------------------------------------------------------------------ blocks with a short side <= 128
// One cluster per block runs everything: momentum, norm, iterations, update or output.
constexpr int kSmallStackSide = 128;     // longest short side
constexpr int kSmallStackSlab = 512;     // columns of a CTA's slab at most
constexpr int kSmallStackItems = 48;    // of a launch: parameters are limited to 32 KB
struct alignas(64) SmallStackItem {
    CUtensorMap map_g, map_m, map_w;   // where `vec` says that TMA moves the array
    const void* G;
    float* M;             // nullable: orthogonalisation alone
    void* W;              // W <- decay * W + step * X; without M: W <- step * X
    long long g_stride, m_stride, w_stride;
    int g_ld, m_ld, w_ld;
    int count, block0;
    int at;               // place of the first block in the class's saved planes
    int g_dtype, w_dtype;
    int vec;              // bit 0: G, bit 1: M, bit 2: W go by TMA
    float decay, step;
};
struct SmallStackIter {
    float zs;             // X^ = fp16(zs * Z)
    float ga, diag;       // fp16 A = ga * Gram - diag on the diagonal
    float pb, pc;         // B~ = pb * A + pc * A^2
};
struct alignas(64) SmallStackClass {
    CUtensorMap x, a, b;  // saved planes: X^_t (turned so that it is wide), A_t, B~_t in slot t of `saved` blocks
    float* info;          // kStackInfo floats per saved block
    int saved;            // 0: nothing is kept
    float f0;             // X_0 = f0 * X^_0
    SmallStackIter it[32];
    int rows, cols, cluster, slab, iters;   // slab: a multiple of 64, cluster * slab >= long side
    int pack;             // 1: two blocks of an item (short side <= 64) to a cluster, in rows 0 .. and 64 ..
    float unit, out;      // Z_0 = unit * X_0; X_T = out * Z
    float beta, eps;
    int nesterov;
    const float* gscale;
    unsigned* status;
};
// The reverse pass of blocks whose iterates were kept, on chip as well: G is the gradient of the output, W
// receives that of the input (no M, step = 1).
constexpr int kSmallGradSlab = 256;      // columns of a CTA's slab at most
struct SmallGradIter {
    float d;              // D^ = fp16(d * V), V = 2^k dL/dX_{t+1}
    float s;              // S^ = s * (D^ X^T + X^ D^T)
    float pa, pb;         // P^ = pa * (S^ A + A S^) + pb * S^
    float va, vb;         // V <- va * V + vb * (B D^ + P^ X^)
};
struct alignas(64) SmallGradClass {
    CUtensorMap x, a, b;
    const float* info;
    int saved;
    SmallGradIter it[32];
    int rows, cols, cluster, slab, iters;
    int pack;             // as above
    float eps;
    unsigned* status;
};
cudaError_t stack_small_grad_launch(const SmallStackItem* items, int n, const SmallGradClass& k, cudaStream_t stream);
// Fills the item's maps and `vec` from its arrays; pack as in the class.
void small_stack_maps(SmallStackItem& it, int rows, int cols, bool pack);
// Clusters of 1, 2, 4 or 8 CTAs that run at once on the current device (they do not fill it: 14 of 8, not 18).
int stack_small_resident(int cluster);
cudaError_t stack_small_launch(const SmallStackItem* items, int n, const SmallStackClass& k, cudaStream_t stream);

}  // namespace muon

// C entry points of the stacked-block operators, the global gradient norm and AdamW: argument
// checks, scales, workspace layout and launches.
//
// Blocks of one shape, whatever stack they come from, form a class: their planes lie one behind the
// other in the workspace and one operation of a chain (stack_chain.cu) covers them.  An iteration is three
// operations per class (Gram, polynomial, apply); tall blocks are not transposed (their Gram matrix is
// X^T X and the apply step X B).
//
// Scales.  With S_t a bound of the singular values of X_t, computed from the schedule (S_0 = 1), the
// planes hold  X_t * tau_t,  A_t * alpha_t,  B_t * gamma_t  with powers of two such that no element
// can leave fp16's range (an element is at most the spectral norm) and ordinary ones keep all 11
// bits: tau ~ sqrt(s) (rows of X_t have norm about 1), alpha ~ r / prod a^2 (A's mean diagonal for a
// flat spectrum).  In the reverse pass an iteration can make the gradient max |p'| times as long (the
// operator norm of the derivative of a matrix function of an odd polynomial p).  The product of these maxima
// is a bound that no gradient keeps up with: they lie at different singular values, so it grows by 1.9 (a
// converging schedule) or 5 (the optimizer's) an iteration while the gradient stays about as it is, and planes
// scaled by it run dry: 0.3 off 64 bits after 32 converging iterations, all zero after 16 of the optimizer's.
// So a chain's D_t is scaled from the measured norm of D_{t+1} and one iteration's bound (GradScale), block by block.
// On chip D is held in fp32, and delta_t scales only the rounded copy that is multiplied; there the bound
// decides whether the block goes that way (kMostGrowth).
//
// Shift.  For a converging schedule the Gram matrix is stored as A - l I with l = sigma_t^2, sigma_t the
// iterates of a flat spectrum (l -> 1): bA + cA^2 = (b + 2cl)(A - lI) + c(A - lI)^2 + (bl + cl^2) I, and the
// last term joins a.  Where X nears its polar factor the stored matrices near zero and their roundings
// vanish with them: a near-orthogonal 96 x 640 block is 5e-5 off 64 bits (2.2e-4 without), the worst case,
// a rank-32 block with noise, 1.8e-4 (1.5e-4).  The optimizer's schedules scatter the singular values over
// 0.7 .. 1.2 and cannot raise tiny ones to 1: there the shift costs accuracy on low-rank blocks (6e-3
// against 8e-4), so they go without.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "adamw.cuh"
#include "runtime.cuh"
#include "stacks.cuh"

namespace muon {
namespace {

constexpr int kMaxSide = 32768;
constexpr long long kMaxBlocks = 1 << 20;
constexpr double kTop = 16384.0;               // no plane's element exceeds this (fp16: 65504)
constexpr double kMaxSigma = 64.0;
constexpr int kMaxTensors = 65536;
// Product of the bounds of |p'| up to which the reverse pass runs on chip.  At 2^18.8 (8 of the optimizer's iterations)
// the scales still cost nothing (128 x 2048 and 96 x 200: the same errors as with measured ones), at 2^19.6 the errors
// of a converging schedule have doubled.
constexpr double kMostGrowth = 524288.0;
// Newton-Schulz planes of one group of blocks; more run group after group in the same space.
constexpr size_t kGroupBytes = static_cast<size_t>(5) << 30;

bool is_dtype(int d) { return d == MUON_BF16 || d == MUON_F32 || d == MUON_F16; }
size_t elem_size(int d) { return d == MUON_F32 ? 4 : 2; }
bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
int up8(int x) { return (x + 7) & ~7; }
double pow2_floor(double x) { return std::exp2(std::floor(std::log2(x))); }

// ---------------------------------------------------------------- schedule
struct Bounds {
    std::vector<double> sigma;    // S_0 .. S_T
    std::vector<double> growth;   // max |p_t'| on [0, S_t]
    std::vector<double> bmax;     // max |b l + c l^2| on [0, S_t^2]
    bool converging = true;       // p_t(1) = 1 and |p_t'(1)| <= 1/2 throughout
    double spread = 1.0;          // product of `growth`
};

// Largest |f| on [0, top] of a function whose interior extrema are among `at`.
template <class F>
double largest(F f, double top, const double* at, int n) {
    double m = std::max(std::fabs(f(0.0)), std::fabs(f(top)));
    for (int i = 0; i < n; ++i)
        if (at[i] > 0.0 && at[i] < top) m = std::max(m, std::fabs(f(at[i])));
    return m;
}

// Whether a gradient through the schedule survives the roundings.  Iterations that neither converge nor repeat (the
// optimizer's scatter the singular values over 0.7 .. 1.2) multiply a rounding of an iterate at every step, and the
// gradient's with it.  For 64 singular values sigma_0 from 1e-2 to 1, with the 11 bits of the operands: e, the error of
// sigma_t, grows by |p'| and gains that of A, B and X; d, that of F = d sigma_t / d sigma_0, grows by |p'| and gains
// |p'' F| e and the reverse pass's own.  A gradient holds the differences (F(x) + F(y)) / (x + y) of all pairs, taken as
// sigma_t / sigma_0, and F itself among about one in a hundred.  Against emulated gradients (96 x 160, the
// optimizer's schedule, hybrids and 30 random ones): estimates up to 0.1 were up to 0.05 off 64 bits, 13 of the
// optimizer's iterations among them (0.09, 0.05); 14 are 0.27 and 0.1, 20 are 6 and 0.6.  Short or calm schedules (five
// of the optimizer's iterations have a spread of 2^11.5) need no estimate.
bool gradient_survives(const muon_ns_schedule& sch, const Bounds& bd) {
    if (bd.spread <= 4096.0) return true;
    constexpr int kPoints = 64;
    const double u2 = std::ldexp(1.0, -22) / 3.0, weight = 0.01;
    double wrong = 0.0, whole = 0.0;
    for (int i = 0; i < kPoints; ++i) {
        const double x0 = std::pow(1e-2, 1.0 - i / (kPoints - 1.0));
        double x = x0, e2 = 0.0, f = 1.0, d2 = 0.0;
        for (int t = 0; t < sch.n_iters; ++t) {
            const double a = sch.coeffs[3 * t], b = sch.coeffs[3 * t + 1], c = sch.coeffs[3 * t + 2];
            const double l = x * x, q = l * (b + c * l), p1 = a + l * (3 * b + 5 * c * l), p2 = x * (6 * b + 20 * c * l);
            const double by_a = l * (b + 2 * c * l);
            d2 = p1 * p1 * d2 + p2 * p2 * f * f * e2 + u2 * f * f * (4 * by_a * by_a + 2 * q * q);
            e2 = p1 * p1 * e2 + u2 * l * (by_a * by_a + 2 * q * q);
            f *= p1;
            x *= a + q;
        }
        wrong += weight * d2 + e2 / (x0 * x0);
        whole += weight * f * f + x * x / (x0 * x0);
    }
    return wrong <= 0.01 * whole;
}

// gradient: one is to come, or this is its call.
muon_status check_schedule(const muon_ns_schedule* s, Bounds& out, bool gradient) {
    if (s == nullptr || s->coeffs == nullptr || s->n_iters < 1 || s->n_iters > MUON_MAX_NS_ITERS)
        return MUON_ERR_INVALID_ARG;
    if (s->fp32_mode != 0 || s->n_split_iters != 0) return MUON_ERR_INVALID_ARG;
    if (!(s->eps > 0.f) || !std::isfinite(s->eps)) return MUON_ERR_INVALID_ARG;
    out.sigma.assign(1, 1.01);
    for (int t = 0; t < s->n_iters; ++t) {
        const double a = s->coeffs[3 * t], b = s->coeffs[3 * t + 1], c = s->coeffs[3 * t + 2];
        if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c)) return MUON_ERR_INVALID_ARG;
        const double top = out.sigma.back(), lam = top * top;
        // p' = a + 3b x + 5c x^2 in x = sigma^2: its roots are p's extrema; p'' vanishes at x = -6b / 20c
        double at[2] = {-1.0, -1.0}, inflect[1] = {-1.0}, vertex[1] = {-1.0};
        if (c != 0.0) {
            const double disc = 9 * b * b - 20 * a * c;
            if (disc >= 0.0) {
                at[0] = (-3 * b + std::sqrt(disc)) / (10 * c);
                at[1] = (-3 * b - std::sqrt(disc)) / (10 * c);
            }
            inflect[0] = -6 * b / (20 * c);
            vertex[0] = -b / (2 * c);
        } else if (b != 0.0) {
            at[0] = -a / (3 * b);
        }
        for (double& x : at) x = x > 0.0 ? std::sqrt(x) : -1.0;
        inflect[0] = inflect[0] > 0.0 ? std::sqrt(inflect[0]) : -1.0;
        auto p = [=](double x) { return x * (a + x * x * (b + c * x * x)); };
        auto dp = [=](double x) { return a + x * x * (3 * b + 5 * c * x * x); };
        auto q = [=](double l) { return l * (b + c * l); };
        if (std::fabs(p(1.0) - 1.0) > 1e-3 || std::fabs(dp(1.0)) > 0.5) out.converging = false;
        out.growth.push_back(std::max(0.25, 1.02 * largest(dp, top, inflect, 1)));
        out.spread *= out.growth.back();
        out.bmax.push_back(std::max(1e-3, largest(q, lam, vertex, 1)));
        const double next = 1.02 * largest(p, top, at, 2) + 0.01;   // room for rounding
        if (!(next <= kMaxSigma)) return MUON_ERR_INVALID_ARG;
        out.sigma.push_back(next);
    }
    return gradient && !gradient_survives(*s, out) ? MUON_ERR_INVALID_ARG : MUON_OK;
}

// ---------------------------------------------------------------- classes of equal blocks
struct StackClass {
    int rows = 0, cols = 0, count = 0;
    int rp = 0, cp = 0, r = 0, s = 0, r8 = 0;   // padded sides; true and padded shorter side
    bool tall = false;
    bool chip = false;                           // iterates on chip, also where its iterates are kept
    bool chip_grad = false;                      // and so does its reverse pass
    int chunks = 0, per = 1;                     // chunks of a block in the elementwise passes
    std::vector<double> alpha, gamma, tau;       // tau[0] unused: X_0 = f0 * plane
    std::vector<double> shift, a, b;             // l; a + bl + cl^2 and b + 2cl (a and b without a shift)
    __half* X = nullptr;                         // x_slots slots: X_t in slot t % x_slots
    __half* L = nullptr;                         // second plane of X_t in slot t & 1
    __half* A = nullptr;                         // a_slots slots: A_t, B_t in slot t % a_slots
    __half* B = nullptr;
    __half* last = nullptr;                      // X_T
    int x_slots = 2, a_slots = 1;
    float* info = nullptr;
    double* partials = nullptr;
    int* done = nullptr;
    size_t plane() const { return static_cast<size_t>(count) * rp * cp * sizeof(__half); }
    size_t square() const { return static_cast<size_t>(count) * r8 * r8 * sizeof(__half); }
};

StackClass make_class(int rows, int cols, const muon_ns_schedule& sch, const Bounds& bd) {
    StackClass c;
    c.rows = rows;
    c.cols = cols;
    c.rp = up8(rows);
    c.cp = up8(cols);
    c.tall = rows > cols;
    c.r = std::min(rows, cols);
    c.s = std::max(rows, cols);
    c.r8 = up8(c.r);
    c.chunks = stack_chunks(c.rp, c.cp, 1);   // at most
    double flat = c.r;   // 1 / (mean diagonal of A_t) for a flat spectrum
    double sigma = 1.0 / std::sqrt(static_cast<double>(c.r));
    for (int t = 0; t < sch.n_iters; ++t) {
        const double lam = bd.sigma[t] * bd.sigma[t];
        c.alpha.push_back(pow2_floor(std::min(std::max(flat, 1.0), kTop / lam)));
        c.gamma.push_back(pow2_floor(std::min(c.alpha.back(), kTop / (2.0 * bd.bmax[t]))));
        const double a = sch.coeffs[3 * t], b = sch.coeffs[3 * t + 1], q = sch.coeffs[3 * t + 2];
        const double l = bd.converging ? sigma * sigma : 0.0;
        c.shift.push_back(l);
        c.a.push_back(a + l * (b + l * q));
        c.b.push_back(b + 2.0 * q * l);
        sigma *= a + sigma * sigma * (b + sigma * sigma * q);
        flat = std::min(flat / std::max(a * a, 1e-6), 1e6);
    }
    const double root = std::exp2(std::round(0.5 * std::log2(static_cast<double>(c.s))));
    for (int t = 0; t <= sch.n_iters; ++t) c.tau.push_back(pow2_floor(std::min(root, kTop / bd.sigma[t])));
    return c;
}

// ---------------------------------------------------------------- classes that run on chip
// Clusters of the on-chip kernels.  As few CTAs as hold the block; more while all blocks' clusters still run at once
// (16 blocks of 96 x 641: 55 us with 4 CTAs each, 98 with 8, of which two do not start before others end; 12 blocks: 57
// and 53).  Up to 256 columns one CTA is faster than several that have to exchange their sums.  Two blocks of up to 64
// rows (or columns) share a cluster where not all run at once (96 of 64 x 2048: 242 us apart, 173 together), or where
// the cluster can be wider then (37 of 64 x 1024: 70 and 55).  pairs: clusters where two blocks of a stack share one.
template <class K>
void set_clusters(K& k, int r, int s, int blocks, int pairs, int most_slab) {
    const int pieces = (s + 63) / 64;
    int least = 1;
    while (least * most_slab < s) least *= 2;
    auto widest = [&](int clusters) {
        int C = least;
        while (s > 256 && 2 * C <= 8 && 2 * C <= pieces && clusters <= stack_small_resident(2 * C)) C *= 2;
        return C;
    };
    int C = widest(blocks);
    k.pack = r <= 64 && (blocks > stack_small_resident(C) || widest(pairs) > C);
    if (k.pack) C = widest(pairs);
    k.cluster = C;
    k.slab = (pieces + C - 1) / C * 64;
}

// The scales of a class whose blocks run in one cluster each (stack_small.cu), or false where they do not:
// a long side above 8 slabs, or a schedule whose product of coefficients a leaves the range in which the
// state's unit keeps X^ and B~ inside fp16.
bool small_class(int rows, int cols, int blocks, int pairs, const muon_ns_schedule& sch, const Bounds& bd, SmallStackClass& k,
                 std::vector<double>* kappas = nullptr) {
    const int r = std::min(rows, cols), s = std::max(rows, cols);
    if (r > kSmallStackSide || s > 8 * kSmallStackSlab) return false;
    const StackClass c = make_class(rows, cols, sch, bd);
    const int T = sch.n_iters;
    double pa = 1.0, top = 1.0;
    for (int t = 0; t < T; ++t) {
        if (!(c.a[t] >= 0.125 && c.a[t] <= 8.0)) return false;
        pa *= c.a[t];
        top = std::max(top, pa);
        if (!(pa >= 1.0 / 65536 && pa <= 65536.0)) return false;
    }
    std::memset(&k, 0, sizeof(k));
    const double tau0 = std::exp2(std::min(14.0, std::round(0.5 * std::log2(static_cast<double>(r) * s))));
    const double unit = pow2_floor(2.0 * top) * c.tau[T] * 16.0;
    pa = 1.0;
    for (int t = 0; t < T; ++t) {
        const double tau = t == 0 ? tau0 : c.tau[t];
        SmallStackIter& f = k.it[t];
        f.zs = static_cast<float>(pa * tau / unit);
        f.ga = static_cast<float>(c.alpha[t] / (tau * tau));
        f.diag = static_cast<float>(c.alpha[t] * c.shift[t]);
        pa *= c.a[t];
        const double kappa = unit / (pa * tau);
        if (!(kappa >= 0.0625 && kappa * 2.0 * bd.bmax[t] <= 2.0 * kTop)) return false;
        if (kappas) kappas->push_back(kappa);
        f.pb = static_cast<float>(kappa * c.b[t] / c.alpha[t]);
        f.pc = static_cast<float>(kappa * sch.coeffs[3 * t + 2] / (c.alpha[t] * c.alpha[t]));
    }
    k.rows = rows;
    k.cols = cols;
    k.iters = T;
    k.unit = static_cast<float>(unit);
    k.out = static_cast<float>(pa / unit);
    k.eps = sch.eps;
    k.f0 = static_cast<float>(1.0 / tau0);
    set_clusters(k, r, s, blocks, pairs, kSmallStackSlab);
    return true;
}

// A run of blocks of one stack inside a group: the class it belongs to and its place there.
struct Part {
    int stack, first, count;   // blocks [first, first + count) of the stack
    int cls, at;               // blocks [at, at + count) of the class
};
struct Group {
    std::vector<StackClass> classes;
    std::vector<Part> parts;
};
struct Shape {
    int count, rows, cols;
    bool small = false;        // runs on chip: takes no part in the groups
};

// The small classes of a call, by shape, and the stacks of each.
struct SmallSet {
    SmallStackClass k;
    std::vector<int> stacks;
};
std::vector<SmallSet> find_small(std::vector<Shape>& shapes, const muon_ns_schedule& sch, const Bounds& bd) {
    std::vector<SmallSet> sets;
    std::vector<std::pair<int, int>> no;
    for (size_t i = 0; i < shapes.size(); ++i) {
        const int rows = shapes[i].rows, cols = shapes[i].cols;
        if (std::min(rows, cols) > kSmallStackSide) continue;
        bool known = false;
        for (SmallSet& s : sets)
            if (s.k.rows == rows && s.k.cols == cols) {
                s.stacks.push_back(static_cast<int>(i));
                shapes[i].small = known = true;
            }
        for (auto& n : no) known = known || (n.first == rows && n.second == cols);
        if (known) continue;
        long long blocks = 0, pairs = 0;
        for (const Shape& s : shapes)
            if (s.rows == rows && s.cols == cols) {
                blocks += s.count;
                pairs += (s.count + 1) / 2;
            }
        SmallSet s;
        if (small_class(rows, cols, static_cast<int>(blocks), static_cast<int>(pairs), sch, bd, s.k)) {
            s.stacks.push_back(static_cast<int>(i));
            shapes[i].small = true;
            sets.push_back(s);
        } else {
            no.push_back({rows, cols});
        }
    }
    return sets;
}

// Cuts the stacks into groups whose planes fit `budget` bytes and whose classes fit one launch.
std::vector<Group> make_groups(const std::vector<Shape>& shapes, const muon_ns_schedule& sch, const Bounds& bd,
                               size_t budget) {
    std::vector<Group> groups(1);
    size_t used = 0;
    for (size_t i = 0; i < shapes.size(); ++i) {
        if (shapes[i].small) continue;
        int first = 0;
        while (first < shapes[i].count) {
            Group* g = &groups.back();
            StackClass one = make_class(shapes[i].rows, shapes[i].cols, sch, bd);
            one.count = 1;
            const size_t each = 4 * one.plane() + 2 * one.square() + static_cast<size_t>(one.chunks) * sizeof(double) +
                                kStackInfo * sizeof(float) + sizeof(int);
            int cls = -1;
            for (size_t k = 0; k < g->classes.size(); ++k)
                if (g->classes[k].rows == one.rows && g->classes[k].cols == one.cols) cls = static_cast<int>(k);
            const size_t room = budget > used ? (budget - used) / each : 0;
            int take = static_cast<int>(std::min<size_t>(shapes[i].count - first, room));
            const bool empty = g->parts.empty();
            if (take == 0 && empty) take = 1;                    // a single block above the budget
            if (take == 0 || (cls < 0 && static_cast<int>(g->classes.size()) == kChainMaxClasses)) {
                groups.emplace_back();
                used = 0;
                continue;
            }
            if (cls < 0) {
                one.count = 0;
                g->classes.push_back(one);
                cls = static_cast<int>(g->classes.size()) - 1;
            }
            StackClass& c = g->classes[cls];
            g->parts.push_back({static_cast<int>(i), first, take, cls, c.count});
            c.count += take;
            used += each * take;
            first += take;
        }
    }
    if (groups.back().parts.empty()) groups.pop_back();
    return groups;
}
// Where iterates are kept for the reverse pass: blocks that run on chip keep them from there, X^ turned so that it
// is wide and B_t scaled as it is there, and their reverse pass runs there too where its slabs hold the block and the
// schedule's bound lets a fixed scale do.  A tall block whose reverse pass runs as a chain has to have X^ as it lies,
// and goes the other way.
void mark_chip(Group& g, const muon_ns_schedule& sch, const Bounds& bd) {
    for (StackClass& c : g.classes) {
        SmallStackClass k;
        std::vector<double> kappas;
        const bool both = c.s <= 8 * kSmallGradSlab && bd.spread <= kMostGrowth;
        if ((c.tall && !both) || !small_class(c.rows, c.cols, c.count, c.count, sch, bd, k, &kappas)) continue;
        c.chip = true;
        c.chip_grad = both;
        c.gamma = kappas;
    }
}

// Pointers of a group's planes; `sv` takes what the reverse pass reads.  Returns the workspace used.  The
// workspace begins with the chain's tile counters.
size_t layout_forward(Group& g, int T, bool saving, Arena& ws, Arena& sv) {
    auto take = [](Arena& a, size_t bytes) { return a.at(a.take(bytes)); };
    take(ws, kStackTickets * sizeof(int));
    for (StackClass& c : g.classes) {
        Arena& keep = saving ? sv : ws;
        c.per = stack_per(c.rp, c.cp, c.count);
        c.chunks = stack_chunks(c.rp, c.cp, c.per);
        c.info = static_cast<float*>(take(keep, static_cast<size_t>(c.count) * kStackInfo * sizeof(float)));
        if (!c.chip) {
            c.partials = static_cast<double*>(take(ws, static_cast<size_t>(c.count) * c.chunks * sizeof(double)));
            c.done = static_cast<int*>(take(ws, static_cast<size_t>(c.count) * sizeof(int)));
        }
        c.x_slots = saving ? T : 2;
        c.a_slots = saving ? T : 1;
        c.X = static_cast<__half*>(take(keep, c.x_slots * c.plane()));
        c.A = static_cast<__half*>(take(keep, c.a_slots * c.square()));
        c.B = static_cast<__half*>(take(keep, c.a_slots * c.square()));
        if (c.chip) continue;
        c.L = static_cast<__half*>(take(ws, 2 * c.plane()));
        if (saving) c.last = static_cast<__half*>(take(ws, c.plane()));
        else c.last = c.X != nullptr ? c.X + (T & 1) * (c.plane() / sizeof(__half)) : nullptr;
    }
    return align_up(ws.used, kAlign);
}

// ---------------------------------------------------------------- chains
// Description of a class for the kernel, and of its operations.
bool chain_class(ChainClass& o, const StackClass& c) {
    std::memset(&o, 0, sizeof(o));
    o.info = c.info;
    o.done = c.done;
    o.rp = c.rp;
    o.cp = c.cp;
    o.r8 = c.r8;
    o.rows = c.rows;
    o.count = c.count;
    const long long pl = static_cast<long long>(c.rp) * c.cp, sq = static_cast<long long>(c.r8) * c.r8;
    o.plane[kPlaneX] = {c.X, pl, c.cp};
    o.plane[kPlaneL] = {c.L, pl, c.cp};
    o.plane[kPlaneA] = {c.A, sq, c.r8};
    o.plane[kPlaneB] = {c.B, sq, c.r8};
    o.plane[kPlaneOut] = {c.last, pl, c.cp};
    const int nx = c.x_slots * c.count, na = c.a_slots * c.count;
    return encode_stack_tmap(&o.map[kMapX], c.X, c.rp, c.cp, nx) && encode_stack_tmap(&o.map[kMapA], c.A, c.r8, c.r8, na) &&
           encode_stack_tmap(&o.map[kMapB], c.B, c.r8, c.r8, na);
}

// Tile width of an operation (in 64 columns): the one whose time is least in this model, in us on a pair of CTAs: a
// 64-deep step of the product takes 0.41, 0.29, 0.24 at 256, 128, 64 columns, the epilogue 4.4 (one plane) or 7 (two
// planes in and out) per 256, and a tile's products overlap the epilogue of the one before.  These are a fit to an
// earlier form of the kernel; its own clock now gives 0.36 and 0.30 for 256 and 64 columns, so narrow tiles are chosen
// somewhat more often than they should be.  2 blocks of 320 x 257: 256 columns make 6 tiles and 13 us per operation, 64
// columns 22 tiles.
int tile_width(const ChainClass& c, ChainOp o, int segments, int pairs) {
    const int kind = o.kind, k = ((kind == 0 ? std::max(c.rp, c.cp) : c.r8) + 63) / 64 * segments;
    const double step[5] = {0.0, 0.24, 0.29, 0.0, 0.41};
    int best = 4;
    double least = 1e30;
    for (int bn : {4, 2, 1}) {
        o.bn = static_cast<uint8_t>(bn);
        const double tiles = static_cast<double>(chain_tiles(c, o)) * c.count, waves = std::ceil(tiles / pairs);
        const double mma = k * step[bn], epi = 0.5 + (kind == 2 ? 7.0 : 4.4) * bn / 4;
        const double t = (waves - 1) * std::max(mma + 0.5, epi) + mma + epi;
        if (t < 0.98 * least) {
            least = t;
            best = bn;
        }
    }
    return best;
}

ChainOp new_op(int cls, int kind, const ChainClass& c, int segments, int pairs) {
    ChainOp o;
    std::memset(&o, 0, sizeof(o));
    o.cls = static_cast<uint8_t>(cls);
    o.kind = static_cast<uint8_t>(kind);
    o.bn = static_cast<uint8_t>(tile_width(c, o, segments, pairs));
    o.e[0] = o.e[1] = o.o[0] = o.o[1] = kPlaneNone;
    return o;
}
void op_e(ChainOp& o, int i, int plane, int slot) {
    o.e[i] = static_cast<uint8_t>(plane);
    o.es[i] = static_cast<uint8_t>(slot);
}
void op_out(ChainOp& o, int i, int plane, int slot) {
    o.o[i] = static_cast<uint8_t>(plane);
    o.os[i] = static_cast<uint8_t>(slot);
}
void op_seg(ChainOp& o, int ma, int sa, int mb, int sb) {
    o.ma[o.nseg] = static_cast<uint8_t>(ma);
    o.sa[o.nseg] = static_cast<uint8_t>(sa);
    o.mb[o.nseg] = static_cast<uint8_t>(mb);
    o.sb[o.nseg] = static_cast<uint8_t>(sb);
    ++o.nseg;
}
struct MapSlot {
    int map, slot;
};
// r x r product of two rows x cols planes over the long side: X Y^T (wide) or X^T Y (tall).
void gram_seg(ChainOp& o, const StackClass& c, MapSlot x, MapSlot y) {
    op_seg(o, x.map, x.slot, y.map, y.slot);
    o.flags = kStackSym | (c.tall ? kStackAMn | kStackBMn : 0u);
}
// r x r product of two symmetric matrices (both read along their rows).
void square_seg(ChainOp& o, int mx, int sx, int my, int sy) {
    op_seg(o, mx, sx, my, sy);
    o.flags = kStackSym;
}
// Symmetric x plane (wide) or plane x symmetric (tall).  Neighbouring tiles share a block of the plane, so that
// the symmetric factor stays in L2.
void apply_seg(ChainOp& o, const StackClass& c, int ms, int ss, MapSlot x) {
    if (c.tall) op_seg(o, x.map, x.slot, ms, ss);
    else op_seg(o, ms, ss, x.map, x.slot);
    o.flags = c.tall ? kStackRowMajor : kStackBMn;
}

struct Call {
    PendingError pending;
    unsigned* status = nullptr;
    cudaStream_t stream = nullptr;
    int sms = 148;
};

// Launches a chain: whole iterations (of `per` operations) at a time, as many as a launch's parameters hold.
muon_status launch_chain(const std::vector<ChainClass>& classes, std::vector<ChainOp>& ops, int per, double flops, int* tickets,
                         const Call& call) {
    // a block's operation starts when all earlier ones of the block are done
    std::vector<int> done(classes.size(), 0);
    for (ChainOp& o : ops) {
        o.need = done[o.cls];
        done[o.cls] += chain_tiles(classes[o.cls], o) * kChainWarps;
    }
    const int all = static_cast<int>(ops.size()), step = std::max(1, kChainMaxOps / per) * per;
    for (int i = 0, k = 0; i < all; i += step, ++k) {
        const int n = std::min(step, all - i);
        const cudaError_t e = launch_timed(MUON_KERNEL_NS_GEMM, flops * n / all, call.stream, [&](cudaStream_t st) {
            return stack_chain_launch(classes.data(), static_cast<int>(classes.size()), ops.data() + i, n, tickets + k,
                                      call.status, call.sms, st);
        });
        if (e != cudaSuccess) return cuda_error(e, "stack chain launch");
    }
    return MUON_OK;
}
muon_status launch_small(const std::vector<SmallStackItem>& items, const SmallStackClass& k, double flops, const Call& call) {
    const cudaError_t e = launch_timed(MUON_KERNEL_NS_GEMM, flops, call.stream, [&](cudaStream_t st) {
        return stack_small_launch(items.data(), static_cast<int>(items.size()), k, st);
    });
    return e == cudaSuccess ? MUON_OK : cuda_error(e, "small-block launch");
}
double small_flops(const SmallStackClass& k, double blocks) {
    const double r = std::min(k.rows, k.cols), s = std::max(k.rows, k.cols);
    return blocks * k.iters * (3.0 * r * r * s + r * r * r);
}
// Clears the status word ahead of the small launches (the passes of a group clear it themselves).
muon_status clear_status(const Call& call) {
    const cudaError_t e = cudaMemsetAsync(call.status, 0, sizeof(unsigned), call.stream);
    return e == cudaSuccess ? MUON_OK : cuda_error(e, "status clear");
}

muon_status launch_pass(StackPass pass, std::vector<StackItem>& items, const StackPassArgs& args, int kind, double bytes,
                        const Call& call) {
    const cudaError_t e = launch_timed(kind, bytes, call.stream, [&](cudaStream_t st) {
        return stack_pass_launch(pass, items.data(), static_cast<int>(items.size()), args, st);
    });
    return e == cudaSuccess ? MUON_OK : cuda_error(e, "stack pass launch");
}

// Class order of the launches: the longest sums first, so that the last tiles are short ones.
std::vector<int> class_order(const Group& g, bool reverse) {
    std::vector<int> o;
    for (size_t i = 0; i < g.classes.size(); ++i)
        if (!(reverse ? g.classes[i].chip_grad : g.classes[i].chip)) o.push_back(static_cast<int>(i));
    std::stable_sort(o.begin(), o.end(), [&](int x, int y) { return g.classes[x].s > g.classes[y].s; });
    return o;
}

// The iterations of a group.  `direct[k]` (if set) receives class k's X_T in bf16 or fp16 instead of
// its plane.
struct Direct {
    void* p = nullptr;
    int ld = 0, dtype = 0;
    long long stride = 0;
};
muon_status run_iterations(Group& g, const muon_ns_schedule& sch, const std::vector<Direct>& direct, int* tickets,
                           const Call& call) {
    const int T = sch.n_iters;
    const std::vector<int> order = class_order(g, false);
    std::vector<ChainClass> classes(g.classes.size());
    for (size_t k = 0; k < classes.size(); ++k) {
        if (g.classes[k].chip) continue;
        if (!chain_class(classes[k], g.classes[k]))
            return cuda_error(cudaErrorInvalidValue, "cuTensorMapEncodeTiled of a stack plane");
        if (direct[k].p != nullptr)
            classes[k].plane[kPlaneOut] = {static_cast<__half*>(direct[k].p), direct[k].stride, direct[k].ld};
        else
            classes[k].rows = g.classes[k].rp;
    }
    std::vector<ChainOp> ops;
    double flops = 0.0;
    for (int t = 0; t < T; ++t) {
        const double cc = sch.coeffs[3 * t + 2];
        for (int stage = 0; stage < 3; ++stage) {
            for (int k : order) {
                const StackClass& c = g.classes[k];
                const double a = c.a[t], b = c.b[t];
                const int xs = t % c.x_slots, as = t % c.a_slots;
                const MapSlot x = {kMapX, xs};
                ChainOp o = new_op(k, stage, classes[k], 1, call.sms / 2);
                if (stage == 0) {
                    gram_seg(o, c, x, x);
                    op_out(o, 0, kPlaneA, as);
                    o.alpha = static_cast<float>(t == 0 ? c.alpha[0] : c.alpha[t] / (c.tau[t] * c.tau[t]));
                    o.diag = static_cast<float>(c.alpha[t] * c.shift[t]);
                    o.pow = t == 0 ? 2 : 0;
                    flops += static_cast<double>(c.count) * c.r * c.r * c.s;
                } else if (stage == 1) {
                    square_seg(o, kMapA, as, kMapA, as);
                    op_e(o, 0, kPlaneA, as);
                    op_out(o, 0, kPlaneB, as);
                    o.alpha = static_cast<float>(cc * c.gamma[t] / (c.alpha[t] * c.alpha[t]));
                    o.beta = static_cast<float>(b * c.gamma[t] / c.alpha[t]);
                    flops += static_cast<double>(c.count) * c.r * c.r * c.r;
                } else {
                    apply_seg(o, c, kMapB, as, x);
                    op_e(o, 0, kPlaneX, xs);
                    op_e(o, 1, kPlaneL, t & 1);
                    double up = c.tau[t + 1];
                    if (t + 1 == T) {
                        op_out(o, 0, kPlaneOut, 0);
                        if (direct[k].p != nullptr) {
                            if (direct[k].dtype == MUON_BF16) o.flags |= kStackOutBf16;
                            up = 1.0;
                        }
                    } else {
                        op_out(o, 0, kPlaneX, (t + 1) % c.x_slots);
                        op_out(o, 1, kPlaneL, (t + 1) & 1);
                    }
                    const double down = t == 0 ? 1.0 : c.tau[t];
                    o.alpha = static_cast<float>(up / (c.gamma[t] * down));
                    o.beta = static_cast<float>(a * up / down);
                    o.pow = t == 0 ? 1 : 0;
                    flops += 2.0 * c.count * c.r * c.r * c.s;
                }
                ops.push_back(o);
            }
        }
    }
    return launch_chain(classes, ops, 3 * static_cast<int>(order.size()), flops, tickets, call);
}

// ---------------------------------------------------------------- arguments
// The arrays that are written: blocks one behind the other, or side by side within a row pitch.
bool blocks_apart(int count, int rows, int cols, int ld, long long stride) {
    if (count <= 1) return true;
    const long long span = static_cast<long long>(rows - 1) * ld + cols;
    if (stride >= span) return true;
    return stride >= cols && (static_cast<long long>(count) - 1) * stride + cols <= ld;
}

muon_status check_view(const void* p, int dtype, int count, int rows, int cols, int ld, long long stride, bool written) {
    if (p == nullptr || !is_dtype(dtype)) return MUON_ERR_INVALID_ARG;
    if (count <= 0 || rows <= 0 || cols <= 0 || stride < 0 || ld < 0) return MUON_ERR_INVALID_ARG;
    if (rows > kMaxSide || cols > kMaxSide || count > kMaxBlocks) return MUON_ERR_UNSUPPORTED_SHAPE;
    if (rows > 1 && ld < cols) return MUON_ERR_INVALID_ARG;
    if (written && !blocks_apart(count, rows, cols, rows > 1 ? ld : cols, stride)) return MUON_ERR_INVALID_ARG;
    if (!aligned_to(p, elem_size(dtype))) return MUON_ERR_ALIGNMENT;
    return MUON_OK;
}

// 8-element vector accesses: base, row pitch and block stride are multiples of 16 bytes.
bool vec_ok(const void* p, int dtype, int ld, long long stride) {
    const int per16 = 16 / static_cast<int>(elem_size(dtype));
    return aligned_to(p, 16) && ld % per16 == 0 && stride % per16 == 0;
}

muon_status check_total(const std::vector<Shape>& shapes) {
    long long blocks = 0;
    for (const Shape& s : shapes) blocks += s.count;
    return blocks > kMaxBlocks ? MUON_ERR_UNSUPPORTED_SHAPE : MUON_OK;
}

muon_status check_stacks(const ns_stack_desc* d, int n, std::vector<Shape>& shapes) {
    if (d == nullptr || n <= 0 || n > kMaxBlocks) return MUON_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i) {
        muon_status st = check_view(d[i].X, d[i].x_dtype, d[i].count, d[i].rows, d[i].cols, d[i].x_ld, d[i].x_stride, false);
        if (st == MUON_OK)
            st = check_view(d[i].Y, d[i].y_dtype, d[i].count, d[i].rows, d[i].cols, d[i].y_ld, d[i].y_stride, true);
        if (st != MUON_OK) return st;
        shapes.push_back({d[i].count, d[i].rows, d[i].cols});
    }
    return check_total(shapes);
}

muon_status check_muon(const muon_stack_desc* d, int n, const muon_hyper* hp, std::vector<Shape>& shapes, Bounds& bd) {
    if (d == nullptr || hp == nullptr || n <= 0 || n > kMaxBlocks) return MUON_ERR_INVALID_ARG;
    muon_status st = check_schedule(&hp->ns, bd, false);
    if (st != MUON_OK) return st;
    if (!std::isfinite(hp->lr) || !std::isfinite(hp->beta) || !std::isfinite(hp->weight_decay)) return MUON_ERR_INVALID_ARG;
    if (hp->nesterov != 0 && hp->nesterov != 1) return MUON_ERR_INVALID_ARG;
    if (hp->scale_mode < MUON_SCALE_MOONLIGHT || hp->scale_mode > MUON_SCALE_NAIVE) return MUON_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i) {
        const muon_stack_desc& s = d[i];
        st = check_view(s.W, s.w_dtype, s.count, s.rows, s.cols, s.w_ld, s.w_stride, true);
        if (st == MUON_OK) st = check_view(s.G, s.g_dtype, s.count, s.rows, s.cols, s.g_ld, s.g_stride, false);
        if (st == MUON_OK) st = check_view(s.M, MUON_F32, s.count, s.rows, s.cols, s.m_ld, s.m_stride, true);
        if (st != MUON_OK) return st;
        shapes.push_back({s.count, s.rows, s.cols});
    }
    return check_total(shapes);
}

double shape_scale(int rows, int cols, int mode) {
    const double o = rows, i = cols;
    switch (mode) {
        case MUON_SCALE_MOONLIGHT: return 0.2 * std::sqrt(std::max(o, i));
        case MUON_SCALE_KJ: return std::sqrt(std::max(1.0, o / i));
        case MUON_SCALE_MUP: return std::sqrt(o / i);
        default: return 1.0;
    }
}

// ---------------------------------------------------------------- layouts
size_t forward_bytes(const std::vector<Shape>& shapes, const muon_ns_schedule& sch, const Bounds& bd, bool saving,
                     size_t* saved) {
    size_t most = 0, kept = 0;
    for (Group& g : make_groups(shapes, sch, bd, saving ? SIZE_MAX : kGroupBytes)) {
        Arena ws, sv;
        sv.used = kept;
        if (saving) mark_chip(g, sch, bd);
        most = std::max(most, layout_forward(g, sch.n_iters, saving, ws, sv));
        kept = align_up(sv.used, kAlign);
    }
    if (saved) *saved = kept;
    return kHeaderBytes + most;
}

// Planes of the reverse pass of a group: D_t and its second plane in slot t & 1.
struct GradPlanes {
    __half* D;
    __half* DL;
    __half* S;
    __half* P;
    float* info;
    double* partials;
    int* done;
    GradScale* scale;
};
std::vector<GradPlanes> layout_backward(const Group& g, int T, Arena& ws) {
    std::vector<GradPlanes> out;
    auto take = [&](size_t bytes) { return ws.at(ws.take(bytes)); };
    take(kStackTickets * sizeof(int));
    for (const StackClass& c : g.classes) {
        GradPlanes p = {};
        if (c.chip_grad) {
            out.push_back(p);
            continue;
        }
        p.info = static_cast<float*>(take(static_cast<size_t>(c.count) * kStackInfo * sizeof(float)));
        p.partials = static_cast<double*>(take(static_cast<size_t>(c.count) * c.chunks * sizeof(double)));
        p.done = static_cast<int*>(take(static_cast<size_t>(c.count) * sizeof(int)));
        p.scale = static_cast<GradScale*>(take(static_cast<size_t>(c.count) * (T + 1) * sizeof(GradScale)));
        p.D = static_cast<__half*>(take(2 * c.plane()));
        p.DL = static_cast<__half*>(take(2 * c.plane()));
        p.S = static_cast<__half*>(take(c.square()));
        p.P = static_cast<__half*>(take(c.square()));
        out.push_back(p);
    }
    return out;
}
size_t backward_bytes(const std::vector<Shape>& shapes, const muon_ns_schedule& sch, const Bounds& bd) {
    size_t most = 0;
    for (Group& g : make_groups(shapes, sch, bd, SIZE_MAX)) {
        Arena ws, fw, sv;
        mark_chip(g, sch, bd);
        layout_forward(g, sch.n_iters, true, fw, sv);
        layout_backward(g, sch.n_iters, ws);
        most = std::max(most, align_up(ws.used, kAlign));
    }
    return kHeaderBytes + most;
}

StackItem base_item(const StackClass& c, const Part& p) {
    StackItem it;
    std::memset(&it, 0, sizeof(it));
    it.rows = c.rows;
    it.cols = c.cols;
    it.count = p.count;
    it.chunks = c.chunks;
    it.per = c.per;
    it.info = c.info + static_cast<size_t>(p.at) * kStackInfo;
    it.partials = c.partials + static_cast<size_t>(p.at) * c.chunks;
    return it;
}
// The chain's counters are the first thing in the workspace after the status word.
int* tickets_at(void* workspace) { return reinterpret_cast<int*>(static_cast<uint8_t*>(workspace) + kHeaderBytes); }
size_t plane_at(const StackClass& c, const Part& p) { return static_cast<size_t>(p.at) * c.rp * c.cp; }

const uint8_t* bytes_at(const void* p, long long blocks, long long stride, int dtype) {
    return static_cast<const uint8_t*>(p) + static_cast<size_t>(blocks) * stride * elem_size(dtype);
}

// ---------------------------------------------------------------- forward
int pairs_of(const Group& g, int cls) {
    int pairs = 0;
    for (const Part& p : g.parts)
        if (p.cls == cls) pairs += (p.count + 1) / 2;
    return pairs;
}
SmallStackItem small_item(const ns_stack_desc& s, int first, int count, bool pack) {
    SmallStackItem it;
    std::memset(&it, 0, sizeof(it));
    it.G = bytes_at(s.X, first, s.x_stride, s.x_dtype);
    it.W = const_cast<uint8_t*>(bytes_at(s.Y, first, s.y_stride, s.y_dtype));
    it.g_stride = s.x_stride;
    it.w_stride = s.y_stride;
    it.g_ld = s.x_ld;
    it.w_ld = s.y_ld;
    it.g_dtype = s.x_dtype;
    it.w_dtype = s.y_dtype;
    it.count = count;
    it.step = 1.f;
    small_stack_maps(it, s.rows, s.cols, pack);
    return it;
}
template <class K>
bool kept_maps(K& q, const StackClass& c, int n) {
    return encode_stack_tmap(&q.x, c.X, std::min(c.rp, c.cp), std::max(c.rp, c.cp), n) &&
           encode_stack_tmap(&q.a, c.A, c.r8, c.r8, n) && encode_stack_tmap(&q.b, c.B, c.r8, c.r8, n);
}
// The on-chip classes of a group whose iterates are kept.
muon_status keep_on_chip(Group& g, const ns_stack_desc* d, const muon_ns_schedule& sch, const Bounds& bd, const Call& call) {
    for (size_t k = 0; k < g.classes.size(); ++k) {
        const StackClass& c = g.classes[k];
        if (!c.chip) continue;
        SmallStackClass q;
        if (!small_class(c.rows, c.cols, c.count, pairs_of(g, static_cast<int>(k)), sch, bd, q)) return MUON_ERR_INVALID_ARG;
        const int n = sch.n_iters * c.count;
        if (!kept_maps(q, c, n)) return cuda_error(cudaErrorInvalidValue, "cuTensorMapEncodeTiled of a stack plane");
        q.info = c.info;
        q.saved = c.count;
        q.status = call.status;
        std::vector<SmallStackItem> items;
        for (const Part& p : g.parts) {
            if (p.cls != static_cast<int>(k)) continue;
            items.push_back(small_item(d[p.stack], p.first, p.count, q.pack != 0));
            items.back().at = p.at;
        }
        const muon_status st = launch_small(items, q, small_flops(q, c.count), call);
        if (st != MUON_OK) return st;
    }
    return MUON_OK;
}

// The reverse pass of the on-chip classes of a group; delta as in backward().
muon_status reverse_on_chip(Group& g, const ns_stack_desc* d, const muon_ns_schedule& sch,
                            const std::vector<std::vector<double>>& delta, const Call& call) {
    for (size_t k = 0; k < g.classes.size(); ++k) {
        const StackClass& c = g.classes[k];
        if (!c.chip_grad) continue;
        const int T = sch.n_iters, n = T * c.count;
        SmallGradClass q;
        std::memset(&q, 0, sizeof(q));
        if (!kept_maps(q, c, n)) return cuda_error(cudaErrorInvalidValue, "cuTensorMapEncodeTiled of a stack plane");
        for (int t = 0; t < T; ++t) {
            const double inv_tau = t == 0 ? 1.0 : 1.0 / c.tau[t], p = 2.0 * c.gamma[t] * inv_tau;   // t = 0: f0 comes from info
            SmallGradIter& f = q.it[t];
            f.d = static_cast<float>(delta[k][t + 1]);
            f.s = static_cast<float>(0.5 * inv_tau);
            f.pa = static_cast<float>(sch.coeffs[3 * t + 2] * p / c.alpha[t]);
            f.pb = static_cast<float>(c.b[t] * p);
            f.va = static_cast<float>(c.a[t]);
            f.vb = static_cast<float>(1.0 / (c.gamma[t] * delta[k][t + 1]));
        }
        q.info = c.info;
        q.saved = c.count;
        q.rows = c.rows;
        q.cols = c.cols;
        q.iters = T;
        q.eps = sch.eps;
        q.status = call.status;
        set_clusters(q, c.r, c.s, c.count, pairs_of(g, static_cast<int>(k)), kSmallGradSlab);
        std::vector<SmallStackItem> items;
        for (const Part& p : g.parts) {
            if (p.cls != static_cast<int>(k)) continue;
            items.push_back(small_item(d[p.stack], p.first, p.count, q.pack != 0));
            items.back().at = p.at;
        }
        const double flops = static_cast<double>(c.count) * T * (6.0 * c.r * c.r * c.s + 2.0 * c.r * c.r * c.r);
        const cudaError_t e = launch_timed(MUON_KERNEL_NS_GEMM, flops, call.stream, [&](cudaStream_t st) {
            return stack_small_grad_launch(items.data(), static_cast<int>(items.size()), q, st);
        });
        if (e != cudaSuccess) return cuda_error(e, "small-block reverse launch");
    }
    return MUON_OK;
}

muon_status orthogonalize(const ns_stack_desc* d, const std::vector<Shape>& shapes, std::vector<SmallSet>& small,
                          const muon_ns_schedule& sch, const Bounds& bd, void* saved, void* workspace, const Call& call) {
    const bool saving = saved != nullptr;
    const int T = sch.n_iters;
    size_t kept = 0;
    bool first = true;
    if (!small.empty()) {
        const muon_status st = clear_status(call);
        if (st != MUON_OK) return st;
        first = false;
    }
    for (SmallSet& set : small) {
        std::vector<SmallStackItem> items;
        double blocks = 0.0;
        for (int i : set.stacks) {
            items.push_back(small_item(d[i], 0, d[i].count, set.k.pack != 0));
            blocks += d[i].count;
        }
        set.k.status = call.status;
        const muon_status st = launch_small(items, set.k, small_flops(set.k, blocks), call);
        if (st != MUON_OK) return st;
    }
    for (Group& g : make_groups(shapes, sch, bd, saving ? SIZE_MAX : kGroupBytes)) {
        Arena ws, sv;
        ws.base = static_cast<uint8_t*>(workspace) + kHeaderBytes;
        sv.base = static_cast<uint8_t*>(saved);
        sv.used = kept;
        if (saving) mark_chip(g, sch, bd);
        layout_forward(g, T, saving, ws, sv);
        kept = align_up(sv.used, kAlign);
        bool any_chip = false;
        for (const StackClass& c : g.classes) any_chip = any_chip || c.chip;
        if (any_chip) {
            muon_status st = MUON_OK;
            if (first) st = clear_status(call);
            first = false;
            if (st == MUON_OK) st = keep_on_chip(g, d, sch, bd, call);
            if (st != MUON_OK) return st;
        }
        std::vector<Direct> direct(g.classes.size());
        std::vector<int> parts_of(g.classes.size(), 0);
        for (const Part& p : g.parts) ++parts_of[p.cls];
        std::vector<StackItem> in, out;
        double read = 0.0, written = 0.0;
        for (const Part& p : g.parts) {
            const StackClass& c = g.classes[p.cls];
            if (c.chip) continue;
            const ns_stack_desc& s = d[p.stack];
            StackItem it = base_item(c, p);
            const double n = static_cast<double>(p.count) * c.rows * c.cols;
            it.G = bytes_at(s.X, p.first, s.x_stride, s.x_dtype);
            it.g_stride = s.x_stride;
            it.g_ld = s.x_ld;
            it.g_dtype = s.x_dtype;
            it.vec = vec_ok(it.G, s.x_dtype, s.x_ld, s.x_stride) ? 1 : 0;
            it.hi = c.X + plane_at(c, p);
            it.lo = c.L + plane_at(c, p);
            it.done = c.done + p.at;
            in.push_back(it);
            read += n * elem_size(s.x_dtype);
            StackItem o = base_item(c, p);
            o.W = const_cast<uint8_t*>(bytes_at(s.Y, p.first, s.y_stride, s.y_dtype));
            o.w_stride = s.y_stride;
            o.w_ld = s.y_ld;
            o.w_dtype = s.y_dtype;
            o.vec = vec_ok(o.W, s.y_dtype, s.y_ld, s.y_stride) ? 4 : 0;
            o.hi = c.last + plane_at(c, p);
            o.step = static_cast<float>(1.0 / c.tau[T]);
            // The last product writes a 16-bit result where it belongs, if one stack is the whole class
            // and its rows are whole 16-byte pieces.
            if (parts_of[p.cls] == 1 && s.y_dtype != MUON_F32 && c.cols % 8 == 0 && o.vec) {
                direct[p.cls] = {o.W, s.y_ld, s.y_dtype, s.y_stride};
            } else {
                out.push_back(o);
                written += n * elem_size(s.y_dtype);
            }
        }
        if (in.empty()) continue;
        StackPassArgs args = {};
        args.eps = sch.eps;
        args.status = first ? call.status : nullptr;
        args.tickets = tickets_at(workspace);
        muon_status st = launch_pass(StackPass::kNorm, in, args, MUON_KERNEL_SCALE, read, call);
        if (st != MUON_OK) return st;
        args.status = call.status;
        st = launch_pass(StackPass::kPack, in, args, MUON_KERNEL_MOMENTUM, 2 * read, call);
        if (st != MUON_OK) return st;
        st = run_iterations(g, sch, direct, args.tickets, call);
        if (st != MUON_OK) return st;
        if (!out.empty()) {
            st = launch_pass(StackPass::kOut, out, args, MUON_KERNEL_MISC, 2 * written, call);
            if (st != MUON_OK) return st;
        }
        first = false;
    }
    return MUON_OK;
}

// ---------------------------------------------------------------- reverse pass
muon_status backward(const ns_stack_desc* d, const std::vector<Shape>& shapes, const muon_ns_schedule& sch,
                     const Bounds& bd, const void* saved, void* workspace, const Call& call) {
    const int T = sch.n_iters;
    size_t kept = 0;
    bool first = true;
    for (Group& g : make_groups(shapes, sch, bd, SIZE_MAX)) {
        Arena ws, sv, fw;
        ws.base = static_cast<uint8_t*>(workspace) + kHeaderBytes;
        sv.base = static_cast<uint8_t*>(const_cast<void*>(saved));
        sv.used = kept;
        mark_chip(g, sch, bd);
        layout_forward(g, T, true, fw, sv);   // the saved planes' places
        kept = align_up(sv.used, kAlign);
        std::vector<GradPlanes> gp = layout_backward(g, T, ws);
        const std::vector<int> order = class_order(g, true);
        const size_t nc = g.classes.size();

        // room[k][t]: how far D_t may reach so that nothing formed from it leaves fp16's range; delta[k][t]: a factor
        // that keeps it there whatever the iterations before have done
        std::vector<std::vector<double>> delta(nc, std::vector<double>(T + 1)), room = delta;
        for (size_t k = 0; k < nc; ++k) {
            const StackClass& c = g.classes[k];
            double nu = 1.0;   // bound of |D_t| relative to the incoming gradient
            for (int t = T; t >= 0; --t) {
                double most = 1.0;
                if (t > 0) {
                    const int u = t - 1;
                    const double lam = bd.sigma[u] * bd.sigma[u];
                    const double inv_tau = u == 0 ? 2.0 / std::sqrt(static_cast<double>(c.rows) * c.cols) : 1.0 / c.tau[u];
                    const double pf = 2.0 * c.gamma[u] * inv_tau * bd.sigma[u] *
                                      (std::fabs(c.b[u]) + 2.0 * std::fabs(sch.coeffs[3 * u + 2]) * lam);
                    most = std::max({1.0, bd.sigma[u], pf});
                }
                room[k][t] = kTop / most;
                delta[k][t] = pow2_floor(room[k][t] / nu);
                if (t > 0) nu *= bd.growth[t - 1];
            }
        }

        bool any_chip = false;
        for (const StackClass& c : g.classes) any_chip = any_chip || c.chip_grad;
        if (any_chip) {
            muon_status st = MUON_OK;
            if (first) st = clear_status(call);
            first = false;
            if (st == MUON_OK) st = reverse_on_chip(g, d, sch, delta, call);
            if (st != MUON_OK) return st;
        }

        std::vector<StackItem> in, dot, out;
        double read = 0.0;
        for (const Part& p : g.parts) {
            const StackClass& c = g.classes[p.cls];
            if (c.chip_grad) continue;
            const GradPlanes& q = gp[p.cls];
            const ns_stack_desc& s = d[p.stack];
            StackItem it = base_item(c, p);
            it.partials = q.partials + static_cast<size_t>(p.at) * c.chunks;
            StackItem o = it;
            it.info = q.info + static_cast<size_t>(p.at) * kStackInfo;
            it.G = bytes_at(s.X, p.first, s.x_stride, s.x_dtype);
            it.g_stride = s.x_stride;
            it.g_ld = s.x_ld;
            it.g_dtype = s.x_dtype;
            it.vec = vec_ok(it.G, s.x_dtype, s.x_ld, s.x_stride) ? 1 : 0;
            const size_t slot = c.plane() / sizeof(__half);
            it.hi = q.D + (T & 1) * slot + plane_at(c, p);
            it.lo = q.DL + (T & 1) * slot + plane_at(c, p);
            it.done = q.done + p.at;
            it.scale = q.scale + static_cast<size_t>(p.at) * (T + 1);
            it.step = static_cast<float>(delta[p.cls][T]);
            in.push_back(it);
            read += static_cast<double>(p.count) * c.rows * c.cols * elem_size(s.x_dtype);
            o.scale = it.scale;
            o.ginfo = it.info;
            o.hi = q.D + plane_at(c, p);
            o.lo = q.DL + plane_at(c, p);
            o.hi2 = c.X + plane_at(c, p);
            o.W = const_cast<uint8_t*>(bytes_at(s.Y, p.first, s.y_stride, s.y_dtype));
            o.w_stride = s.y_stride;
            o.w_ld = s.y_ld;
            o.w_dtype = s.y_dtype;
            o.vec = vec_ok(o.W, s.y_dtype, s.y_ld, s.y_stride) ? 4 : 0;
            out.push_back(o);
        }
        if (in.empty()) continue;
        StackPassArgs args = {};
        args.eps = sch.eps;
        args.status = first ? call.status : nullptr;
        args.tickets = tickets_at(workspace);
        args.iters = T;
        muon_status st = launch_pass(StackPass::kNorm, in, args, MUON_KERNEL_SCALE, read, call);
        if (st != MUON_OK) return st;
        args.status = call.status;
        st = launch_pass(StackPass::kPackGrad, in, args, MUON_KERNEL_MOMENTUM, 2 * read, call);
        if (st != MUON_OK) return st;

        std::vector<ChainClass> classes(nc);
        for (size_t k = 0; k < nc; ++k) {
            const StackClass& c = g.classes[k];
            const GradPlanes& q = gp[k];
            ChainClass& o = classes[k];
            if (c.chip_grad) continue;
            const long long pl = static_cast<long long>(c.rp) * c.cp, sq = static_cast<long long>(c.r8) * c.r8;
            const bool ok = chain_class(o, c) && encode_stack_tmap(&o.map[kMapD], q.D, c.rp, c.cp, 2 * c.count) &&
                            encode_stack_tmap(&o.map[kMapS], q.S, c.r8, c.r8, c.count) &&
                            encode_stack_tmap(&o.map[kMapP], q.P, c.r8, c.r8, c.count);
            if (!ok) return cuda_error(cudaErrorInvalidValue, "cuTensorMapEncodeTiled of a stack plane");
            o.done = q.done;
            o.scale = q.scale;
            o.scales = T + 1;
            o.plane[kPlaneD] = {q.D, pl, c.cp};
            o.plane[kPlaneDL] = {q.DL, pl, c.cp};
            o.plane[kPlaneS] = {q.S, sq, c.r8};
            o.plane[kPlaneP] = {q.P, sq, c.r8};
        }
        std::vector<ChainOp> ops;
        double flops = 0.0;
        for (int t = T - 1; t >= 0; --t) {
            const double cc = sch.coeffs[3 * t + 2];
            const MapSlot x = {kMapX, t}, dd = {kMapD, (t + 1) & 1};
            for (int stage = 0; stage < 3; ++stage) {
                for (int k : order) {
                    const StackClass& c = g.classes[k];
                    const double a = c.a[t], b = c.b[t];
                    const double inv_tau = t == 0 ? 1.0 : 1.0 / c.tau[t];   // t = 0: f0 comes from info
                    ChainOp o = new_op(k, stage, classes[k], 2, call.sms / 2);
                    if (stage == 0) {          // S = (D X^T + X D^T) / 2
                        gram_seg(o, c, dd, x);
                        gram_seg(o, c, x, dd);
                        op_out(o, 0, kPlaneS, 0);
                        o.alpha = static_cast<float>(0.5 * inv_tau);
                        flops += 2.0 * c.count * c.r * c.r * c.s;
                    } else if (stage == 1) {   // P * 2 gamma / tau, P = bS + c(SA + AS)
                        square_seg(o, kMapS, 0, kMapA, t);
                        square_seg(o, kMapA, t, kMapS, 0);
                        op_e(o, 0, kPlaneS, 0);
                        op_out(o, 0, kPlaneP, 0);
                        o.alpha = static_cast<float>(cc * 2.0 * c.gamma[t] * inv_tau / c.alpha[t]);
                        o.beta = static_cast<float>(b * 2.0 * c.gamma[t] * inv_tau);
                        flops += 2.0 * c.count * c.r * c.r * c.r;
                    } else {                   // D' = aD + BD + 2PX
                        apply_seg(o, c, kMapB, t, dd);
                        apply_seg(o, c, kMapP, 0, x);
                        op_e(o, 0, kPlaneD, (t + 1) & 1);
                        op_e(o, 1, kPlaneDL, (t + 1) & 1);
                        op_out(o, 0, kPlaneD, t & 1);
                        op_out(o, 1, kPlaneDL, t & 1);
                        o.flags |= kStackRescale;
                        o.t = static_cast<uint8_t>(t);
                        o.room = static_cast<float>(room[k][t] / bd.growth[t]);
                        o.alpha = static_cast<float>(1.0 / c.gamma[t]);
                        o.beta = static_cast<float>(a);
                        flops += 4.0 * c.count * c.r * c.r * c.s;
                    }
                    if (t == 0 && stage < 2) o.pow = 1;
                    ops.push_back(o);
                }
            }
        }
        st = launch_chain(classes, ops, 3 * static_cast<int>(order.size()), flops, args.tickets, call);
        if (st != MUON_OK) return st;
        dot = out;
        st = launch_pass(StackPass::kDot, dot, args, MUON_KERNEL_SCALE, 0.0, call);
        if (st != MUON_OK) return st;
        st = launch_pass(StackPass::kGradOut, out, args, MUON_KERNEL_MISC, 2 * read, call);
        if (st != MUON_OK) return st;
        first = false;
    }
    return MUON_OK;
}

// ---------------------------------------------------------------- Muon step
int step_vec(const muon_stack_desc& s) {
    return (vec_ok(s.G, s.g_dtype, s.g_ld, s.g_stride) ? 1 : 0) | (vec_ok(s.M, MUON_F32, s.m_ld, s.m_stride) ? 2 : 0) |
           (vec_ok(s.W, s.w_dtype, s.w_ld, s.w_stride) ? 4 : 0);
}

muon_status step(const muon_stack_desc* d, const std::vector<Shape>& shapes, std::vector<SmallSet>& small,
                 const muon_hyper& hp, const Bounds& bd, const float* grad_scale, void* workspace, const Call& call) {
    const int T = hp.ns.n_iters;
    bool first = true;
    if (!small.empty()) {
        const muon_status st = clear_status(call);
        if (st != MUON_OK) return st;
        first = false;
    }
    for (SmallSet& set : small) {
        std::vector<SmallStackItem> items;
        double blocks = 0.0;
        for (int i : set.stacks) {
            const muon_stack_desc& s = d[i];
            SmallStackItem it;
            std::memset(&it, 0, sizeof(it));
            it.G = s.G;
            it.M = s.M;
            it.W = s.W;
            it.g_stride = s.g_stride; it.m_stride = s.m_stride; it.w_stride = s.w_stride;
            it.g_ld = s.g_ld; it.m_ld = s.m_ld; it.w_ld = s.w_ld;
            it.g_dtype = s.g_dtype;
            it.w_dtype = s.w_dtype;
            it.count = s.count;
            it.decay = static_cast<float>(1.0 - static_cast<double>(hp.lr) * hp.weight_decay);
            it.step = static_cast<float>(-static_cast<double>(hp.lr) * shape_scale(s.rows, s.cols, hp.scale_mode));
            small_stack_maps(it, s.rows, s.cols, set.k.pack != 0);
            items.push_back(it);
            blocks += s.count;
        }
        set.k.beta = hp.beta;
        set.k.nesterov = hp.nesterov;
        set.k.gscale = grad_scale;
        set.k.status = call.status;
        const muon_status st = launch_small(items, set.k, small_flops(set.k, blocks), call);
        if (st != MUON_OK) return st;
    }
    for (Group& g : make_groups(shapes, hp.ns, bd, kGroupBytes)) {
        Arena ws, sv;
        ws.base = static_cast<uint8_t*>(workspace) + kHeaderBytes;
        layout_forward(g, T, false, ws, sv);
        std::vector<StackItem> in, out;
        double norm_bytes = 0.0, pack_bytes = 0.0, upd_bytes = 0.0;
        for (const Part& p : g.parts) {
            const StackClass& c = g.classes[p.cls];
            const muon_stack_desc& s = d[p.stack];
            StackItem it = base_item(c, p);
            it.G = bytes_at(s.G, p.first, s.g_stride, s.g_dtype);
            it.M = reinterpret_cast<float*>(const_cast<uint8_t*>(bytes_at(s.M, p.first, s.m_stride, MUON_F32)));
            it.W = const_cast<uint8_t*>(bytes_at(s.W, p.first, s.w_stride, s.w_dtype));
            it.g_stride = s.g_stride; it.m_stride = s.m_stride; it.w_stride = s.w_stride;
            it.g_ld = s.g_ld; it.m_ld = s.m_ld; it.w_ld = s.w_ld;
            it.g_dtype = s.g_dtype; it.w_dtype = s.w_dtype;
            it.vec = step_vec(s);   // a later first block keeps it: its offset is a multiple of the stride
            it.hi = c.X + plane_at(c, p);
            it.lo = c.L + plane_at(c, p);
            it.done = c.done + p.at;
            in.push_back(it);
            it.hi = c.last + plane_at(c, p);
            it.decay = static_cast<float>(1.0 - static_cast<double>(hp.lr) * hp.weight_decay);
            it.step = static_cast<float>(-static_cast<double>(hp.lr) * shape_scale(c.rows, c.cols, hp.scale_mode) / c.tau[T]);
            out.push_back(it);
            const double n = static_cast<double>(p.count) * c.rows * c.cols;
            norm_bytes += n * (elem_size(s.g_dtype) + 8.0);
            pack_bytes += n * ((hp.nesterov ? elem_size(s.g_dtype) : 0.0) + 8.0);
            upd_bytes += n * (2.0 * elem_size(s.w_dtype) + 2.0);
        }
        StackPassArgs args = {};
        args.eps = hp.ns.eps;
        args.beta = hp.beta;
        args.nesterov = hp.nesterov;
        args.gscale = grad_scale;
        args.status = first ? call.status : nullptr;
        args.tickets = tickets_at(workspace);
        muon_status st = launch_pass(StackPass::kNorm, in, args, MUON_KERNEL_MOMENTUM, norm_bytes, call);
        if (st != MUON_OK) return st;
        args.status = call.status;
        st = launch_pass(StackPass::kPack, in, args, MUON_KERNEL_MISC, pack_bytes, call);
        if (st != MUON_OK) return st;
        st = run_iterations(g, hp.ns, std::vector<Direct>(g.classes.size()), args.tickets, call);
        if (st != MUON_OK) return st;
        st = launch_pass(StackPass::kUpdate, out, args, MUON_KERNEL_UPDATE, upd_bytes, call);
        if (st != MUON_OK) return st;
        first = false;
    }
    return MUON_OK;
}

muon_status make_call(Call& call, void* workspace, void* stream) {
    call.status = static_cast<unsigned*>(workspace);
    call.stream = static_cast<cudaStream_t>(stream);
    call.sms = device_sm_count();
    return MUON_OK;
}

// ---------------------------------------------------------------- norm, AdamW
muon_status check_tensors(const adamw_tensor_desc* d, int n, bool all) {
    if (d == nullptr || n <= 0 || n > kMaxTensors) return MUON_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i) {
        const adamw_tensor_desc& t = d[i];
        if (t.n < 0 || !is_dtype(t.g_dtype) || (all && !is_dtype(t.w_dtype))) return MUON_ERR_INVALID_ARG;
        if (t.n == 0) continue;
        if (t.G == nullptr || (all && (t.W == nullptr || t.m == nullptr || t.v == nullptr))) return MUON_ERR_INVALID_ARG;
        if (!aligned_to(t.G, elem_size(t.g_dtype))) return MUON_ERR_ALIGNMENT;
        if (all && (!aligned_to(t.W, elem_size(t.w_dtype)) || !aligned_to(t.m, 4) || !aligned_to(t.v, 4)))
            return MUON_ERR_ALIGNMENT;
    }
    return MUON_OK;
}
std::vector<AdamItem> adam_items(const adamw_tensor_desc* d, int n) {
    std::vector<AdamItem> items;
    items.reserve(n);
    for (int i = 0; i < n; ++i) {
        if (d[i].n == 0) continue;
        AdamItem it;
        std::memset(&it, 0, sizeof(it));
        it.W = d[i].W; it.G = d[i].G; it.m = d[i].m; it.v = d[i].v;
        it.n = d[i].n;
        it.w_dtype = d[i].w_dtype; it.g_dtype = d[i].g_dtype;
        it.vec = (aligned_to(it.G, 16) ? 1 : 0) | (aligned_to(it.m, 16) && aligned_to(it.v, 16) ? 2 : 0) |
                 (aligned_to(it.W, 16) ? 4 : 0);
        items.push_back(it);
    }
    return items;
}
constexpr int kMostSms = 256;   // the norm's partials: room for any device of this architecture
size_t norm_bytes(int n) {
    const size_t launches = (static_cast<size_t>(n) + kAdamMaxItems - 1) / kAdamMaxItems;
    return kHeaderBytes + align_up(launches * kMostSms * kAdamCtasPerSm * sizeof(double), kAlign);
}

}  // namespace

namespace {
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encode_fn() {
    static const EncodeFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}
// A map of `count` matrices (strides in elements): boxes of 128 bytes x box_rows rows of one matrix, 128-byte
// swizzle, zeros outside.
bool encode_map(CUtensorMap* out, const void* base, CUtensorMapDataType type, int es, int rows, int cols, int count,
                long long ld, long long stride, int box_rows) {
    const EncodeFn fn = encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t gdim[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(count)};
    const cuuint64_t gstride[2] = {static_cast<cuuint64_t>(ld) * es, static_cast<cuuint64_t>(stride) * es};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / es), static_cast<cuuint32_t>(box_rows), 1u};
    const cuuint32_t estride[3] = {1u, 1u, 1u};
    return fn(out, type, 3, const_cast<void*>(base), gdim, gstride, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
}  // namespace

bool encode_stack_tmap(CUtensorMap* out, const void* base, int rows, int cols, int count) {
    return encode_map(out, base, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, rows, cols, count, cols,
                      static_cast<long long>(rows) * cols, 64);
}

void small_stack_maps(SmallStackItem& it, int rows, int cols, bool pack) {
    it.vec = 0;
    auto one = [&](CUtensorMap& m, int bit, const void* p, int dtype, int ld, long long stride) {
        if (p == nullptr) return;
        // a map's strides are positive: single rows and single blocks get the dense ones
        const long long per16 = 16 / static_cast<long long>(elem_size(dtype));
        const long long l = rows > 1 ? ld : cols;
        const long long t = it.count > 1 ? stride : l * rows;
        // Rows are whole 16-byte pieces: a store's clipping at the row's end is no finer (measured: a row of one
        // fp16 came out four long).  Blocks whose rows interleave have legal maps too.
        if (!aligned_to(p, 16) || cols % per16 != 0 || l % per16 != 0 || t % per16 != 0 || l <= 0 || t <= 0) return;
        const CUtensorMapDataType type = dtype == MUON_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                         : dtype == MUON_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                             : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
        // what the encoder refuses goes element by element
        if (encode_map(&m, p, type, static_cast<int>(elem_size(dtype)), rows, cols, it.count, l, t, rows > cols || pack ? 64 : 128))
            it.vec |= bit;
    };
    one(it.map_g, 1, it.G, it.g_dtype, it.g_ld, it.g_stride);
    one(it.map_m, 2, it.M, MUON_F32, it.m_ld, it.m_stride);
    one(it.map_w, 4, it.W, it.w_dtype, it.w_ld, it.w_stride);
}

}  // namespace muon

using namespace muon;

extern "C" {

size_t ns_stacks_workspace_size(const ns_stack_desc* descs, int n, const muon_ns_schedule* sch, int with_saved) {
    size_t bytes = 0;
    no_throw([&] {
        std::vector<Shape> shapes;
        Bounds bd;
        muon_status st = check_schedule(sch, bd, with_saved != 0);
        if (st == MUON_OK) st = check_stacks(descs, n, shapes);
        if (st == MUON_OK && !with_saved) find_small(shapes, *sch, bd);
        if (st == MUON_OK) bytes = forward_bytes(shapes, *sch, bd, with_saved != 0, nullptr);
        return st;
    });
    return bytes;
}

size_t ns_stacks_saved_size(const ns_stack_desc* descs, int n, const muon_ns_schedule* sch) {
    size_t bytes = 0;
    no_throw([&] {
        std::vector<Shape> shapes;
        Bounds bd;
        muon_status st = check_schedule(sch, bd, true);
        if (st == MUON_OK) st = check_stacks(descs, n, shapes);
        if (st == MUON_OK) forward_bytes(shapes, *sch, bd, true, &bytes);
        return st;
    });
    return bytes;
}

muon_status ns_orthogonalize_stacks(const ns_stack_desc* descs, int n, const muon_ns_schedule* sch, void* saved,
                                    size_t saved_bytes, void* workspace, size_t ws_bytes, void* stream) {
    return no_throw([&] {
        std::vector<Shape> shapes;
        Bounds bd;
        muon_status st = check_schedule(sch, bd, saved != nullptr);
        if (st == MUON_OK) st = check_stacks(descs, n, shapes);
        if (st != MUON_OK) return st;
        if (workspace == nullptr) return MUON_ERR_INVALID_ARG;
        if (!aligned_to(workspace, 256) || !aligned_to(saved, 256)) return MUON_ERR_ALIGNMENT;
        size_t kept = 0;
        std::vector<SmallSet> small;   // the reverse pass reads what only the grouped launches keep
        if (saved == nullptr) small = find_small(shapes, *sch, bd);
        const size_t need = forward_bytes(shapes, *sch, bd, saved != nullptr, &kept);
        if (ws_bytes < need || (saved != nullptr && saved_bytes < kept)) return MUON_ERR_WORKSPACE_TOO_SMALL;
        Call call;
        st = make_call(call, workspace, stream);
        if (st != MUON_OK) return st;
        return orthogonalize(descs, shapes, small, *sch, bd, saved, workspace, call);
    });
}

size_t ns_stacks_backward_workspace_size(const ns_stack_desc* descs, int n, const muon_ns_schedule* sch) {
    size_t bytes = 0;
    no_throw([&] {
        std::vector<Shape> shapes;
        Bounds bd;
        muon_status st = check_schedule(sch, bd, true);
        if (st == MUON_OK) st = check_stacks(descs, n, shapes);
        if (st == MUON_OK) bytes = backward_bytes(shapes, *sch, bd);
        return st;
    });
    return bytes;
}

muon_status ns_orthogonalize_stacks_backward(const ns_stack_desc* descs, int n, const muon_ns_schedule* sch,
                                             const void* saved, size_t saved_bytes, void* workspace, size_t ws_bytes,
                                             void* stream) {
    return no_throw([&] {
        std::vector<Shape> shapes;
        Bounds bd;
        muon_status st = check_schedule(sch, bd, true);
        if (st == MUON_OK) st = check_stacks(descs, n, shapes);
        if (st != MUON_OK) return st;
        if (workspace == nullptr || saved == nullptr) return MUON_ERR_INVALID_ARG;
        if (!aligned_to(workspace, 256) || !aligned_to(saved, 256)) return MUON_ERR_ALIGNMENT;
        size_t kept = 0;
        forward_bytes(shapes, *sch, bd, true, &kept);
        if (saved_bytes < kept || ws_bytes < backward_bytes(shapes, *sch, bd)) return MUON_ERR_WORKSPACE_TOO_SMALL;
        Call call;
        st = make_call(call, workspace, stream);
        if (st != MUON_OK) return st;
        return backward(descs, shapes, *sch, bd, saved, workspace, call);
    });
}

size_t muon_stacks_workspace_size(const muon_stack_desc* descs, int n, const muon_hyper* hp) {
    size_t bytes = 0;
    no_throw([&] {
        std::vector<Shape> shapes;
        Bounds bd;
        const muon_status st = check_muon(descs, n, hp, shapes, bd);
        if (st == MUON_OK) {
            find_small(shapes, hp->ns, bd);
            bytes = forward_bytes(shapes, hp->ns, bd, false, nullptr);
        }
        return st;
    });
    return bytes;
}

muon_status muon_step_stacks(const muon_stack_desc* descs, int n, const muon_hyper* hp, const float* grad_scale,
                             void* workspace, size_t ws_bytes, void* stream) {
    return no_throw([&] {
        std::vector<Shape> shapes;
        Bounds bd;
        muon_status st = check_muon(descs, n, hp, shapes, bd);
        if (st != MUON_OK) return st;
        if (workspace == nullptr) return MUON_ERR_INVALID_ARG;
        if (!aligned_to(workspace, 256) || !aligned_to(grad_scale, 4)) return MUON_ERR_ALIGNMENT;
        std::vector<SmallSet> small = find_small(shapes, hp->ns, bd);
        if (ws_bytes < forward_bytes(shapes, hp->ns, bd, false, nullptr)) return MUON_ERR_WORKSPACE_TOO_SMALL;
        Call call;
        st = make_call(call, workspace, stream);
        if (st != MUON_OK) return st;
        return step(descs, shapes, small, *hp, bd, grad_scale, workspace, call);
    });
}

size_t grad_norm_workspace_size(const adamw_tensor_desc* descs, int n) {
    return check_tensors(descs, n, false) == MUON_OK ? norm_bytes(n) : 0;
}

muon_status grad_norm_batched(const adamw_tensor_desc* descs, int n, float max_norm, float* out, void* workspace,
                              size_t ws_bytes, void* stream) {
    return no_throw([&] {
        muon_status st = check_tensors(descs, n, false);
        if (st != MUON_OK) return st;
        if (out == nullptr || workspace == nullptr || !(max_norm > 0.f)) return MUON_ERR_INVALID_ARG;
        if (!aligned_to(out, 4) || !aligned_to(workspace, 256)) return MUON_ERR_ALIGNMENT;
        if (ws_bytes < norm_bytes(n)) return MUON_ERR_WORKSPACE_TOO_SMALL;
        Call call;
        st = make_call(call, workspace, stream);
        if (st != MUON_OK) return st;
        const std::vector<AdamItem> items = adam_items(descs, n);
        double* partials = reinterpret_cast<double*>(static_cast<uint8_t*>(workspace) + kHeaderBytes);
        double bytes = 0.0;
        for (const AdamItem& it : items) bytes += static_cast<double>(it.n) * elem_size(it.g_dtype);
        const cudaError_t e = launch_timed(MUON_KERNEL_GRAD_NORM, bytes, call.stream, [&](cudaStream_t s) {
            return grad_norm_launch(items.data(), static_cast<int>(items.size()), partials, max_norm, out, call.status,
                                    std::min(call.sms, kMostSms), s);
        });
        return e == cudaSuccess ? MUON_OK : cuda_error(e, "gradient norm launch");
    });
}

muon_status adamw_step_batched(const adamw_tensor_desc* descs, int n, const adamw_hyper* hp, const float* grad_scale,
                               void* stream) {
    return no_throw([&] {
        muon_status st = check_tensors(descs, n, true);
        if (st != MUON_OK) return st;
        if (hp == nullptr || !std::isfinite(hp->lr) || !std::isfinite(hp->weight_decay)) return MUON_ERR_INVALID_ARG;
        if (!(hp->beta1 >= 0.0 && hp->beta1 < 1.0) || !(hp->beta2 >= 0.0 && hp->beta2 < 1.0)) return MUON_ERR_INVALID_ARG;
        if (!(hp->eps >= 0.0) || !std::isfinite(hp->eps)) return MUON_ERR_INVALID_ARG;
        if (hp->step_dev == nullptr && hp->step < 1) return MUON_ERR_INVALID_ARG;
        if (!aligned_to(grad_scale, 4) || !aligned_to(hp->step_dev, 8)) return MUON_ERR_ALIGNMENT;
        const std::vector<AdamItem> items = adam_items(descs, n);
        AdamParams p = {};
        const double t = static_cast<double>(hp->step);
        p.lr = static_cast<float>(hp->lr);
        p.beta1 = static_cast<float>(hp->beta1);
        p.beta2 = static_cast<float>(hp->beta2);
        p.omb1 = static_cast<float>(1.0 - hp->beta1);
        p.omb2 = static_cast<float>(1.0 - hp->beta2);
        p.eps = static_cast<float>(hp->eps);
        p.decay = static_cast<float>(1.0 - hp->lr * hp->weight_decay);
        p.beta1_d = hp->beta1;
        p.beta2_d = hp->beta2;
        if (hp->step_dev == nullptr) {
            p.c1 = static_cast<float>(1.0 / (1.0 - std::pow(p.beta1_d, t)));
            p.c2 = static_cast<float>(1.0 / (1.0 - std::pow(p.beta2_d, t)));
        }
        p.step = hp->step_dev;
        p.gscale = grad_scale;
        double bytes = 0.0;
        for (const AdamItem& it : items)
            bytes += static_cast<double>(it.n) * (elem_size(it.g_dtype) + 2.0 * elem_size(it.w_dtype) + 16.0);
        const PendingError pending;
        const int sms = device_sm_count();
        const cudaError_t e = launch_timed(MUON_KERNEL_ADAMW, bytes, static_cast<cudaStream_t>(stream), [&](cudaStream_t s) {
            return adamw_launch(items.data(), static_cast<int>(items.size()), p, sms, s);
        });
        return e == cudaSuccess ? MUON_OK : cuda_error(e, "AdamW launch");
    });
}

}  // extern "C"

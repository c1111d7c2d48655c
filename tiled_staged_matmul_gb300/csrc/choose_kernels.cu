// choose_kernels.cu -- the choice of experts and its gradient.
//
//   s = softmax(x) or sigmoid(x) over a token's logits x;  c = s + bias
//   groups of experts are kept by the sum of their one or two largest c, then
//   the topk largest c of the kept groups are chosen;  ties go to the lower number
//   w_j = s[id_j] (/ sum_j s[id_j]) * scale
//
//   g_j = scale dw_j, or scale / S (dw_j - sum_i dw_i s_i / S) with S = sum_i s_i
//   dx = s (ds - sum ds s) for the softmax, ds s (1 - s) for the sigmoid, ds_e = sum of
//   the g_j with id_j = e
//
// A warp takes a token.  Scores are formed in f32, but which expert is chosen is
// what it is in f64: where two scores that decide something lie within the bound
// of their f32 errors, the warp forms them again in f64 and decides by those.  What
// f64 rounds alike (with a bias the sigmoids of 40 and 45) goes to the lower number.
// (Without a bias the logits themselves give the order, exactly.)  With random
// logits one token in a thousand needs it.
//
// Bound by instructions rather than by its bytes.  So the choice is not made one
// expert after another (370 instructions for 8 of 256) but among few: the topk-th
// largest of the lanes' maxima bounds the topk-th largest of all from below, a
// dozen experts reach it, and those move to a lane each and are ranked there
// (8192 x 256, 8 of 4 of 8 groups, with a bias: 14 us, 28.8 one after another;
// without groups 12, without a bias either 8 to 9, of 1024 in bf16 18 to 19).  Where the
// largest lie together in few lanes there are too many candidates, and they are taken one
// after another after all (scores in the order of the experts' numbers: 30).  So they
// are for every token where the kept groups' lanes are no more than topk (with a bias)
// and hold more than 32 experts: 8 of 2 of 8 groups 32 us, by the softmax 41; and with a
// bias for choices near 32, a warp's lanes: 31 of 256 56, 32, which leaves none for the
// one that comes next and so ends in f64, 159.  Compiled once per type of the logits
// (-DTSM_CHOOSE_ELEM, gemm_internal.h's kOut* values).
#include "fp4_internal.h"
#include "fp4_ptx.cuh"
#include "launch.cuh"
#include "piece.cuh"

#ifndef TSM_CHOOSE_ELEM
#error "compile with -DTSM_CHOOSE_ELEM=<element type>"
#endif

namespace tsm {

namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kChooseWarps = 4;  // tokens of a block

__device__ __forceinline__ bool is_nan(float v) { return v != v; }

// A float's place in the order of floats, above 0 (which stands for none);
// -0 as +0.
__device__ __forceinline__ uint32_t order_of(float v)
{
    const uint32_t b = __float_as_uint(v + 0.f);
    return b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint64_t order_of(double v)
{
    const uint64_t b = uint64_t(__double_as_longlong(v + 0.0));
    return b ^ (uint64_t(int64_t(b) >> 63) | (uint64_t(1) << 63));
}

// The float with this place in order.
__device__ __forceinline__ float value_of(uint32_t o)
{
    return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}

__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(kAll, v); }
__device__ __forceinline__ uint64_t warp_max(uint64_t v)
{
    const uint32_t hi = __reduce_max_sync(kAll, uint32_t(v >> 32));
    const uint32_t lo = __reduce_max_sync(kAll, uint32_t(v >> 32) == hi ? uint32_t(v) : 0u);
    return (uint64_t(hi) << 32) | lo;
}

template <typename F>
__device__ __forceinline__ F warp_sum(F v)
{
#pragma unroll
    for (int d = 16; d; d >>= 1)
        v += __shfl_xor_sync(kAll, v, d);
    return v;
}

// An order's type.
template <typename F>
struct OrderOf {
    using type = uint32_t;
};
template <>
struct OrderOf<double> {
    using type = uint64_t;
};

// Where a token's experts lie in its warp: L lanes to a group, VM experts to a
// lane, so that lanes and a lane's experts are in ascending order.
struct Layout {
    int group;  // this lane's
    int first;  // this lane's first expert
    int count;  // how many it has
    __device__ __forceinline__ Layout(int per, int groups, int lanes_log, int vm, int lane)
    {
        group = lane >> lanes_log;
        const int at = (lane & ((1 << lanes_log) - 1)) * vm;
        first = group * per + at;
        count = group < groups ? max(0, min(vm, per - at)) : 0;
    }
};

// A lane's logits; -infinity for what it has no expert for.
template <int ET, int VM, bool WIDE>
__device__ __forceinline__ void read_logits(const ChooseParams &p, int64_t token, const Layout &at, float (&x)[VM])
{
    constexpr int EB = ET == kOutF32 ? 4 : 2;
    using E = Piece<ET, EB>;
    const char *row = static_cast<const char *>(p.logits) + (token * p.ld + at.first) * EB;
    if constexpr (WIDE && VM * EB >= 4) {
        // (All of a lane's experts or none are there.)
        using P = Piece<ET, VM * EB >= 16 ? 16 : 4>;
#pragma unroll
        for (int i = 0; i < VM / P::V; ++i) {
            float v[P::V];
#pragma unroll
            for (int j = 0; j < P::V; ++j)
                v[j] = __uint_as_float(0xff800000u);
            if (at.count)
                P::widen(P::get(row, i), v);
#pragma unroll
            for (int j = 0; j < P::V; ++j)
                x[P::V * i + j] = v[j];
        }
    } else {
#pragma unroll
        for (int i = 0; i < VM; ++i) {
            float v[1] = {__uint_as_float(0xff800000u)};
            if (i < at.count)
                E::widen(E::get(row, i), v);
            x[i] = v[0];
        }
    }
}

template <int ET>
__device__ __forceinline__ float logit_at(const ChooseParams &p, int64_t token, int e)
{
    constexpr int EB = ET == kOutF32 ? 4 : 2;
    using E = Piece<ET, EB>;
    float v[1];
    E::widen(E::get(static_cast<const char *>(p.logits) + token * p.ld * EB, e), v);
    return v[0];
}

// Bounds of the f32 error of a score s <= 1.  exp(v) by ex2.approx is off by 2 +
// 1.173 |v| units in the last place at most, which s (1 - s) weighs: (0.5 + 0.27) 2^-23;
// the sum rounds by 2^-24, the division by 2 x 2^-23.  For the softmax the
// exponentials' errors (e^-d (2 + 1.173 d) 2^-23 with d = max - x: 2 x 2^-23), the
// total's (as large, and 40 roundings of 2^-24) and the quotient's: 25 x 2^-23.
constexpr float kSigmoidError = 4.f / 8388608.f, kSoftmaxError = 25.f / 8388608.f;

// A group's sum of one or two values: the sum in f32, and what it may be off by.  Each value
// has its score's error and is rounded, with its bias in it, and so is the sum: by a
// part of the values' sizes, not of the sum's, in which they may cancel.
constexpr float kLargest = 3.402823466e38f;
template <typename F>
struct GroupSum {
    F v = F(0);
    float off = 0.f;
    __device__ __forceinline__ void add(F c, float eps)
    {
        v += c;
        off += eps + 0x1p-22f * fminf(fabsf(float(c)), kLargest);  // (2^-24 each: c, the sum, its bound)
    }
};
// The least (to = -1) or the most (1) that it is in exact arithmetic.  What has left f32's
// range is as far as that goes: two biases' sum may be there, or one of +infinity.
__device__ __forceinline__ float bound_of(float v, float off, float to)
{
    return to * (fmaxf(to * v, -kLargest) + off);
}

// A score in F; `top` and `sum` are the softmax's.
template <typename F>
__device__ __forceinline__ F score_of(bool sigmoid, float x, float top, F sum)
{
    if constexpr (sizeof(F) == 4)
        return sigmoid ? __fdividef(1.f, 1.f + __expf(-x)) : __fdividef(__expf(x - top), sum);
    else
        return sigmoid ? F(1) / (F(1) + exp(-F(x))) : exp(F(x) - F(top)) / sum;
}

// The warp's choice, one expert after another, formed in F.  Lane j ends with the
// j-th chosen expert, -1 where there is none.  False: two f32 values that decide
// something are too close.
template <typename F, int ET, int VM>
__device__ __forceinline__ bool choose_in_turn(const ChooseParams &p, int64_t token, const Layout &at, const float (&x)[VM], float top,
                                       float total, int lane, int &id)
{
    using O = typename OrderOf<F>::type;
    constexpr bool CHECK = sizeof(F) == 4;
    const float none = __uint_as_float(0xff800000u);
    const bool limited = p.keep < p.groups;
    const bool by_score = p.bias || (limited && p.best > 1);
    F sum = F(total);
    if (!CHECK && by_score && !p.sigmoid) {
        F mine = F(0);
#pragma unroll
        for (int i = 0; i < VM; ++i)
            if (x[i] != none)
                mine += exp(F(x[i]) - F(top));
        sum = warp_sum(mine);
    }
    auto score = [&](float v) { return score_of<F>(p.sigmoid, v, top, sum); };
    // Places in order, 0 where there is no expert to choose.
    O c[VM];
#pragma unroll
    for (int i = 0; i < VM; ++i) {
        const float bias = p.bias && i < at.count ? p.bias[at.first + i] : 0.f;
        c[i] = 0;
        if (i < at.count && x[i] != none && bias != none)
            c[i] = order_of(p.bias ? score(x[i]) + F(bias) : F(x[i]));
    }
    auto value_of = [](O o) {  // the number with this place
        if constexpr (sizeof(O) == 4) {
            const uint32_t b = o & 0x80000000u ? o ^ 0x80000000u : ~o;
            return __uint_as_float(b);
        } else {
            const uint64_t b = o >> 63 ? o ^ (uint64_t(1) << 63) : ~o;
            return __longlong_as_double(int64_t(b));
        }
    };
    const float eps = p.sigmoid ? kSigmoidError : kSoftmaxError;
    bool sure = true;
    if (limited) {
        // The group's one or two best: a lane's, then its lanes'.
        O a = 0, b = 0;
        auto take = [&](O v) {
            b = max(b, min(a, v));
            a = max(a, v);
        };
#pragma unroll
        for (int i = 0; i < VM; ++i)
            take(c[i]);
        for (int d = 1; d < (1 << p.lanes_log); d <<= 1) {
            const O a2 = __shfl_xor_sync(kAll, a, d), b2 = __shfl_xor_sync(kAll, b, d);
            b = max(min(a, a2), max(b, b2));
            a = max(a, a2);
        }
        // (Without a bias the places are the logits'.)
        const auto value = [&](O o) { return p.bias || p.best == 1 ? F(value_of(o)) : score(float(value_of(o))); };
        GroupSum<F> sum;
        if (a != 0)
            sum.add(value(a), eps);
        if (p.best > 1 && b != 0)
            sum.add(value(b), eps);
        O g = a == 0 ? O(0) : order_of(sum.v);
        // Lane l < groups holds group l's.
        g = __shfl_sync(kAll, g, min(lane, p.groups - 1) * (1 << p.lanes_log));
        // Its rank among the groups.
        int before = 0;
        for (int j = 0; j < p.groups; ++j) {
            const O other = __shfl_sync(kAll, g, j);
            before += other > g || (other == g && j < lane);
        }
        const bool kept = lane < p.groups && before < p.keep && g != 0;
        if (CHECK && by_score) {
            // No group that is kept may lie below one that is not.
            const float off = __shfl_sync(kAll, sum.off, min(lane, p.groups - 1) * (1 << p.lanes_log));
            const uint32_t edge = g != 0 ? order_of(bound_of(float(value_of(g)), off, kept ? -1.f : 1.f)) : 0u;
            sure = __reduce_min_sync(kAll, kept ? edge : kAll) > warp_max(kept || lane >= p.groups ? 0u : edge);
        }
        const uint32_t mask = __ballot_sync(kAll, kept);
        if (!(mask >> (at.group & 31) & 1u)) {
#pragma unroll
            for (int i = 0; i < VM; ++i)
                c[i] = 0;
        }
    }
    // One after another.  With the check one more than are wanted: the one that
    // comes next.
    O mine = 0, best = 0;
#pragma unroll
    for (int i = 0; i < VM; ++i)
        best = max(best, c[i]);
    id = -1;
    const bool check = CHECK && p.bias;
    const int rounds = min(p.topk + (check ? 1 : 0), 32);
    for (int j = 0; j < rounds; ++j) {
        const O m = warp_max(best);
        if (m == 0)
            break;
        const int winner = __ffs(__ballot_sync(kAll, best == m)) - 1;
        int which = 0;
        if (lane == winner) {
            bool found = false;
            best = 0;
#pragma unroll
            for (int i = 0; i < VM; ++i) {
                if (!found && c[i] == m) {
                    found = true;
                    which = at.first + i;
                    c[i] = 0;
                }
                best = max(best, c[i]);
            }
        }
        which = __shfl_sync(kAll, which, winner);
        if (lane == j) {
            id = which;
            mine = m;
        }
    }
    if (check) {
        const O next = __shfl_down_sync(kAll, mine, 1);
        const float a = float(value_of(mine)), b = float(value_of(next));
        bool close = lane < p.topk && mine != 0 && next != 0 && a - b <= eps * (2.f + fabsf(a) + fabsf(b));
        // Experts alike in logit and bias tie in any arithmetic (but the last one
        // may have more of them after it).
        const float xi = id >= 0 ? logit_at<ET>(p, token, id) : 0.f, bi = id >= 0 ? p.bias[id] : 0.f;
        const float xn = __shfl_down_sync(kAll, xi, 1), bn = __shfl_down_sync(kAll, bi, 1);
        const bool alike = xi == xn && bi == bn;
        close &= !(alike && lane < p.topk - 1);
        // With 32 choices there is no lane for the one that comes next.
        const bool more = warp_max(best) != 0;
        if (lane == 31)
            close = p.topk == 32 && more;
        sure &= __all_sync(kAll, !close) != 0;
    }
    if (lane >= p.topk)
        id = -1;
    return sure;
}

// The one or two largest of a group's lanes' values, in every lane of the group.
template <typename T>
__device__ __forceinline__ void best_of_lanes(T &a, T &b, int lanes)
{
    for (int d = 1; d < lanes; d <<= 1) {
        const T a2 = __shfl_xor_sync(kAll, a, d), b2 = __shfl_xor_sync(kAll, b, d);
        b = max(min(a, a2), max(b, b2));
        a = max(a, a2);
    }
}

// The sum of a group's `best` largest scores (with the bias) in f64, a whole warp
// for one group.  Sigmoids only.
template <int ET>
__device__ __forceinline__ double group_exactly(const ChooseParams &p, int64_t token, int group, int per, int lane)
{
    const double none = __longlong_as_double(0xfff0000000000000ll);
    double a = none, b = none;
    for (int i = lane; i < per; i += 32) {
        const int e = group * per + i;
        const float x = logit_at<ET>(p, token, e), add = p.bias ? p.bias[e] : 0.f;
        if (x == __uint_as_float(0xff800000u) || add == __uint_as_float(0xff800000u))
            continue;
        const double v = score_of<double>(true, x, 0.f, 1.0) + double(add);
        b = fmax(b, fmin(a, v));
        a = fmax(a, v);
    }
    __syncwarp();
    best_of_lanes(a, b, 32);
    return p.best > 1 && b != none ? a + b : a;
}

// The groups that are kept, by it: the sure ones, and the largest of the open ones.
template <int ET>
__device__ __noinline__ uint32_t kept_exactly(const ChooseParams &p, int64_t token, uint32_t sure, uint32_t open)
{
    const int lane = int(threadIdx.x & 31);
    double exact = 0.0;
    for (uint32_t left = open; left; left &= left - 1) {
        const int group = __ffs(left) - 1;
        const double d = group_exactly<ET>(p, token, group, p.per, lane);
        if (lane == group)
            exact = d;
    }
    int rank = 0;
    for (uint32_t left = open; left; left &= left - 1) {
        const int j = __ffs(left) - 1;
        const double other = __shfl_sync(kAll, exact, j);
        rank += other > exact || (other == exact && j < lane);
    }
    return sure | __ballot_sync(kAll, (open >> lane & 1u) && rank < p.keep - __popc(sure));
}

// The rank of a lane's candidate among `n` by its score (a sigmoid) in f64.
template <int ET>
__device__ __noinline__ int rank_exactly(const ChooseParams &p, int64_t token, int name, int n)
{
    const int lane = int(threadIdx.x & 31);
    double exact = 0.0;
    if (lane < n)
        exact = score_of<double>(true, logit_at<ET>(p, token, name), 0.f, 1.0) + double(p.bias[name]);
    __syncwarp();
    int rank = 0;
    for (int j = 0; j < n; ++j) {
        const double other = __shfl_sync(kAll, exact, j);
        rank += other > exact || (other == exact && j < lane);
    }
    return rank;
}

// The warp's choice: as choose_in_turn, for what a warp of candidates holds.  `keys`
// and `names` are the warp's, 32 each.
enum class Chosen { kYes, kInTurn, kExactly };  // done, too many candidates, f64 is needed for all
template <int ET, int VM>
__device__ __forceinline__ Chosen choose(const ChooseParams &p, int64_t token, const Layout &at, const float (&x)[VM], const float (&add)[VM], float top,
                                         float total, int lane, uint32_t *keys, int *names, int &id)
{
    const float none = __uint_as_float(0xff800000u);
    const bool limited = p.keep < p.groups;
    const float eps = p.sigmoid ? kSigmoidError : kSoftmaxError;
    uint32_t c[VM];  // places in order, 0 where there is no expert to choose
    // (What is no expert's has a logit of -infinity.)
    const auto place = [&](auto &&value) {
#pragma unroll
        for (int i = 0; i < VM; ++i)
            c[i] = x[i] == none || add[i] == none ? 0u : order_of(value(i));
    };
    if (!p.bias)
        place([&](int i) { return x[i]; });
    else if (p.sigmoid)
        place([&](int i) { return score_of<float>(true, x[i], top, total) + add[i]; });
    else
        place([&](int i) { return score_of<float>(false, x[i], top, total) + add[i]; });
    if (limited) {
        uint32_t a = 0, b = 0;
#pragma unroll
        for (int i = 0; i < VM; ++i) {
            b = max(b, min(a, c[i]));
            a = max(a, c[i]);
        }
        best_of_lanes(a, b, (1 << p.lanes_log));
        const bool by_score = p.bias || p.best > 1;
        // (Without a bias the places are the logits'.)
        const auto value = [&](uint32_t o) {
            return p.bias || !by_score ? value_of(o) : score_of<float>(p.sigmoid, value_of(o), top, total);
        };
        GroupSum<float> sum;
        if (a != 0)
            sum.add(value(a), eps);
        if (p.best > 1 && b != 0)
            sum.add(value(b), eps);
        uint32_t g = a == 0 ? 0u : order_of(sum.v);
        // Lane l < groups holds group l's; its rank.
        g = __shfl_sync(kAll, g, min(lane, p.groups - 1) * (1 << p.lanes_log));
        int before = 0;
        for (int j = 0; j < p.groups; ++j) {
            const uint32_t other = __shfl_sync(kAll, g, j);
            before += other > g || (other == g && j < lane);
        }
        const bool mine = lane < p.groups && g != 0;
        uint32_t mask = __ballot_sync(kAll, mine && before < p.keep);
        if (by_score) {
            // Those that may lie on the other side of the border between the groups that
            // are kept and those that are not are ranked again in f64.
            const bool kept = mask >> lane & 1u;
            const float off = __shfl_sync(kAll, sum.off, min(lane, p.groups - 1) * (1 << p.lanes_log));
            const uint32_t edge = mine ? order_of(bound_of(value_of(g), off, kept ? -1.f : 1.f)) : 0u;
            const uint32_t least = __reduce_min_sync(kAll, kept ? edge : kAll);
            const uint32_t most = warp_max(kept ? 0u : edge);
            if (least <= most) {
                if (!p.sigmoid)
                    return Chosen::kExactly;
                const uint32_t sure = __ballot_sync(kAll, kept && edge > most);
                const uint32_t open = __ballot_sync(kAll, kept ? edge <= most : edge >= least);
                mask = kept_exactly<ET>(p, token, sure, open);
            }
        }
        if (!(mask >> (at.group & 31) & 1u)) {
#pragma unroll
            for (int i = 0; i < VM; ++i)
                c[i] = 0;
        }
    }
    // At least `want` experts lie at or above the want-th largest of the lanes'
    // maxima (equal ones are taken together).  With a bias one more than are
    // chosen, and what may be as large.
    const bool check = p.bias != nullptr;
    const int want = p.topk + (check ? 1 : 0);
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < VM; ++i)
        best = max(best, c[i]);
    uint32_t low = 1;
    for (int n = 0; n < want;) {
        const uint32_t m = warp_max(best);
        if (m == 0) {
            low = 1;
            break;
        }
        low = m;
        n += __popc(__ballot_sync(kAll, best == m));
        if (best == m)
            best = 0;
    }
    if (check && low > 1) {
        const float v = value_of(low);  // (+infinity with a bias of that: then those alone)
        low = order_of(v - 3.f * eps - 0.25f * eps * fminf(fabsf(v), kLargest));
    }
    int mine = 0;
#pragma unroll
    for (int i = 0; i < VM; ++i)
        mine += c[i] >= low;
    int before = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(kAll, before, d);
        if (lane >= d)
            before += v;
    }
    const int n = __shfl_sync(kAll, before, 31);
    if (n > 32)
        return Chosen::kInTurn;
    before -= mine;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < VM; ++i)
        if (c[i] >= low) {
            keys[before] = c[i];
            names[before++] = at.first + i;
        }
    __syncwarp();
    uint32_t key = lane < n ? keys[lane] : 0u;
    int name = lane < n ? names[lane] : 1 << 30;
    int rank = 0;
    for (int j = 0; j < n; ++j) {
        const uint32_t other = __shfl_sync(kAll, key, j);
        rank += other > key || (other == key && j < lane);  // (candidates are in order of their numbers)
    }
    if (check) {
        // Sorted, is anyone that is chosen too close to the next?
        __syncwarp();
        if (lane < n)
            keys[rank] = key;
        __syncwarp();
        const float a = value_of(key), b = rank + 1 < n ? value_of(keys[rank + 1]) : none;
        const bool close = lane < n && rank < p.topk && rank + 1 < n && !(a - b > 2.f * eps + 0.25f * eps * (fabsf(a) + fabsf(b)));
        if (__any_sync(kAll, close)) {
            if (!p.sigmoid)
                return Chosen::kExactly;
            rank = rank_exactly<ET>(p, token, name, n);
        }
    }
    __syncwarp();
    if (lane < n)
        names[rank] = name;
    __syncwarp();
    id = lane < min(n, p.topk) ? names[lane] : -1;
    return Chosen::kYes;
}

// One after another, in f32 or (as few tokens need) f64; out of the way of the usual
// path's registers.
template <int ET, int VM, bool WIDE>
__device__ __noinline__ int choose_slowly(const ChooseParams &p, int64_t token, float top, float total, bool exactly)
{
    const int lane = int(threadIdx.x & 31);
    const Layout at(p.per, p.groups, p.lanes_log, VM, lane);
    float x[VM];
    read_logits<ET, VM, WIDE>(p, token, at, x);
    int id;
    if (exactly || !choose_in_turn<float, ET, VM>(p, token, at, x, top, total, lane, id))
        choose_in_turn<double, ET, VM>(p, token, at, x, top, total, lane, id);
    return id;
}

template <int ET, int VM, bool WIDE>
__global__ void __launch_bounds__(32 * kChooseWarps, VM == 32 ? 2 : VM == 16 ? 4 : VM == 8 && !WIDE ? 5 : 6) tsm_choose_kernel(const __grid_constant__ ChooseParams p)
{
    chain_next();
    chain_wait();
    __shared__ uint32_t keys[kChooseWarps][32];
    __shared__ int names[kChooseWarps][32];
    const int lane = int(threadIdx.x & 31);
    const Layout at(p.per, p.groups, p.lanes_log, VM, lane);
    const float none = __uint_as_float(0xff800000u);
    // (Fewer than 2^31 tokens, and far fewer warps.)
    for (uint32_t t = blockIdx.x * kChooseWarps + (threadIdx.x >> 5); t < uint32_t(p.tokens); t += gridDim.x * kChooseWarps) {
        float x[VM];
        read_logits<ET, VM, WIDE>(p, t, at, x);
        // (seen: NaN where there is one.  add: the bias.)
        float seen = 0.f, add[VM];
#pragma unroll
        for (int i = 0; i < VM; ++i) {
            add[i] = p.bias && (WIDE ? at.count > 0 : i < at.count) ? p.bias[at.first + i] : 0.f;
            seen = ptx::max_abs3_nan(seen, x[i], add[i]);
        }
        bool bad = is_nan(seen);
        float top = 0.f, total = 1.f;
        if (!p.sigmoid) {
            uint32_t high = 0;
#pragma unroll
            for (int i = 0; i < VM; ++i)
                high = max(high, x[i] != none ? order_of(x[i]) : 0u);
            high = warp_max(high);
            top = high ? value_of(high) : 0.f;
            bad |= top == __uint_as_float(0x7f800000u);
            total = 0.f;
#pragma unroll
            for (int i = 0; i < VM; ++i)
                total += __expf(x[i] - top);
            total = warp_sum(total);
        }
        bad = __any_sync(kAll, bad);
        int id = lane;
        if (!bad) {
            const Chosen how = choose<ET, VM>(p, t, at, x, add, top, total, lane, keys[threadIdx.x >> 5], names[threadIdx.x >> 5], id);
            if (how != Chosen::kYes)
                id = choose_slowly<ET, VM, WIDE>(p, t, top, total, how == Chosen::kExactly);
        }
        if (lane >= p.topk)
            id = -1;
        float w = 0.f;
        const float mine = id >= 0 ? logit_at<ET>(p, t, id) : 0.f;
        if (p.renormalize) {
            // s_j / sum s, with the largest exponential taken out of both.
            const float e = p.sigmoid ? fminf(mine, 0.f) : mine;
            const uint32_t m = warp_max(id >= 0 ? order_of(e) : 0u);
            const float most = m ? value_of(m) : 0.f;
            if (id >= 0)
                w = expf(e - most) / (p.sigmoid ? 1.f + expf(-fabsf(mine)) : 1.f);
            const float all = warp_sum(w);
            w = id >= 0 ? w / all * p.scale : 0.f;
        } else if (id >= 0) {
            w = (p.sigmoid ? 1.f / (1.f + expf(-mine)) : expf(mine - top) / total) * p.scale;
        }
        if (bad)
            w = __uint_as_float(0x7fffffffu);
        if (lane < p.topk) {
            p.ids[int64_t(t) * p.topk + lane] = id;
            p.weights[int64_t(t) * p.topk + lane] = w;
        }
    }
}

template <int ET, int VM, bool WIDE>
__global__ void __launch_bounds__(32 * kChooseWarps) tsm_choose_grad_kernel(const __grid_constant__ ChooseParams p)
{
    constexpr int EB = ET == kOutF32 ? 4 : 2;
    using E = Piece<ET, EB>;
    chain_next();
    chain_wait();
    const int lane = int(threadIdx.x & 31);
    const Layout at(p.experts, 1, 5, VM, lane);
    const bool whole = !p.sigmoid && !p.renormalize;
    const int64_t warps = int64_t(gridDim.x) * kChooseWarps;
    for (int64_t t = int64_t(blockIdx.x) * kChooseWarps + (threadIdx.x >> 5); t < p.tokens; t += warps) {
        int id = lane < p.topk ? p.ids[t * p.topk + lane] : -1;
        if (id >= p.experts || id < 0)
            id = -1;
        const float dw = id >= 0 ? p.dweights[t * p.topk + lane] * p.scale : 0.f;
        const float mine = id >= 0 ? logit_at<ET>(p, t, id) : 0.f;
        float x[VM];
        float top = 0.f, total = 1.f;
        if (whole) {
            read_logits<ET, VM, WIDE>(p, t, at, x);
            float high = __uint_as_float(0xff800000u);
#pragma unroll
            for (int i = 0; i < VM; ++i)
                high = fmaxf(high, x[i]);
            top = high;
#pragma unroll
            for (int d = 16; d; d >>= 1)
                top = fmaxf(top, __shfl_xor_sync(kAll, top, d));
            if (top == __uint_as_float(0xff800000u))
                top = 0.f;  // (no expert is there: zeros below)
            total = 0.f;
#pragma unroll
            for (int i = 0; i < VM; ++i) {
                x[i] = expf(x[i] - top);
                total += x[i];
            }
            total = warp_sum(total);
        }
        // The lane's choice: g_j ds_j/dx_j but for the softmax's sum.
        float g = 0.f, sum = 0.f;
        if (p.renormalize) {
            const float e = p.sigmoid ? fminf(mine, 0.f) : mine;
            const uint32_t m = warp_max(id >= 0 ? order_of(e) : 0u);
            const float most = m ? value_of(m) : 0.f;
            float w = 0.f;
            if (id >= 0)
                w = expf(e - most) / (p.sigmoid ? 1.f + expf(-fabsf(mine)) : 1.f);
            const float all = warp_sum(w);
            w = all > 0.f || is_nan(all) ? w / all : 0.f;
            const float mean = warp_sum(dw * w);
            g = w * (dw - mean) * (p.sigmoid ? 1.f / (1.f + expf(mine)) : 1.f);
        } else if (p.sigmoid) {
            const float s = 1.f / (1.f + expf(-mine));
            g = dw * s * (1.f / (1.f + expf(mine)));
        } else {
            g = dw * (id >= 0 ? expf(mine - top) / total : 0.f);
            sum = warp_sum(g);
        }
        if (id < 0)
            g = 0.f;
        float d[VM];
        const float per = whole && total > 0.f ? sum / total : whole && is_nan(total) ? total : 0.f;
#pragma unroll
        for (int i = 0; i < VM; ++i)
            d[i] = whole ? 0.f - x[i] * per : 0.f;
        char *const first = static_cast<char *>(p.dlogits) + t * p.ld_d * EB;
        char *row = first + at.first * EB;
        if constexpr (WIDE && VM * EB >= 4) {
            using P = Piece<ET, VM * EB >= 16 ? 16 : 4>;
            if (at.count) {
#pragma unroll
                for (int i = 0; i < VM / P::V; ++i) {
                    float v[P::V];
#pragma unroll
                    for (int j = 0; j < P::V; ++j)
                        v[j] = d[P::V * i + j];
                    P::store(row, i, v);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < VM; ++i)
                if (i < at.count) {
                    const float v[1] = {d[i]};
                    E::store(row, i, v);
                }
        }
        // Over these the choices' own, each by its lane; those of one expert by the first
        // of them, in their order.  (8192 x 256 4.2 us, 6.0 with every choice compared with
        // every lane's experts; 8192 x 1024 bf16 10.8 and 16.0.)
        const uint32_t alike = __match_any_sync(kAll, id);
        float v[1] = {whole ? 0.f - expf(mine - top) * per : 0.f};
        if (__any_sync(kAll, id >= 0 && (alike & (alike - 1)) != 0)) {
            for (int j = 0; j < p.topk; ++j) {
                const float other = __shfl_sync(kAll, g, j);
                v[0] += alike >> j & 1u ? other : 0.f;
            }
        } else {
            v[0] += g;
        }
        __syncwarp();
        if (id >= 0 && lane == __ffs(alike) - 1)
            E::store(first, id, v);
    }
}

template <int ET, int VM, bool GRAD>
cudaError_t choose_as(const ChooseParams &p, bool wide, int sms, cudaStream_t stream)
{
    const int64_t blocks = (p.tokens + kChooseWarps - 1) / kChooseWarps;
    const dim3 grid(unsigned(min(blocks, int64_t(sms) * 64)));
    if constexpr (GRAD)
        return wide ? launch_chained(tsm_choose_grad_kernel<ET, VM, true>, grid, 32 * kChooseWarps, 0, 0, stream, p)
                    : launch_chained(tsm_choose_grad_kernel<ET, VM, false>, grid, 32 * kChooseWarps, 0, 0, stream, p);
    else
        return wide ? launch_chained(tsm_choose_kernel<ET, VM, true>, grid, 32 * kChooseWarps, 0, 0, stream, p)
                    : launch_chained(tsm_choose_kernel<ET, VM, false>, grid, 32 * kChooseWarps, 0, 0, stream, p);
}

template <int ET, bool GRAD>
cudaError_t choose_type(ChooseParams p, bool aligned, int sms, cudaStream_t stream)
{
    p.per = p.experts / p.groups;
    for (p.lanes_log = 5; p.groups << p.lanes_log > 32; --p.lanes_log) {
    }
    // Experts of a lane: a power of two that lets a group's lanes hold its experts.
    int vm = 2;
    while (vm << p.lanes_log < p.per)
        vm *= 2;
    // Wide accesses where every lane's experts are all there or all not, and start
    // at a multiple of them.
    const bool wide = aligned && p.per % vm == 0;
    switch (vm) {
    case 2: return choose_as<ET, 2, GRAD>(p, wide, sms, stream);
    case 4: return choose_as<ET, 4, GRAD>(p, wide, sms, stream);
    case 8: return choose_as<ET, 8, GRAD>(p, wide, sms, stream);
    case 16: return choose_as<ET, 16, GRAD>(p, wide, sms, stream);
    case 32: return choose_as<ET, 32, GRAD>(p, wide, sms, stream);
    default: return cudaErrorInvalidValue;  // (more than the caller lets through)
    }
}

}  // namespace

template <>
cudaError_t launch_choose<TSM_CHOOSE_ELEM>(const ChooseParams &p, bool aligned, int sms, cudaStream_t stream)
{
    return choose_type<TSM_CHOOSE_ELEM, false>(p, aligned, sms, stream);
}

template <>
cudaError_t launch_choose_grad<TSM_CHOOSE_ELEM>(const ChooseParams &p, bool aligned, int sms, cudaStream_t stream)
{
    return choose_type<TSM_CHOOSE_ELEM, true>(p, aligned, sms, stream);
}

}  // namespace tsm

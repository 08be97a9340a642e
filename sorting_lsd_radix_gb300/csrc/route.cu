// A router's choice of experts for every token, and its gradient.
//
// Token t's scores are s[e] = softmax_e(l[t]) or sigmoid(l[t][e]); an expert is
// chosen by s[e] + bias[e], or without a bias by the order of its logit, which
// is the score's.  With groups, a group is worth the sum of its one or two best
// choice values, and the best groups' experts alone can be chosen.  The weights
// are the chosen experts' scores without the bias, if asked divided by their
// sum, times a scale.  The gradient of w with respect to l, g = scale * d_w,
// q = w / scale:
//   softmax                p_j * (g_j [j chosen] - sum_k g_k p_k)
//   softmax, renormalised  q_k * (g_k - sum g q) at the chosen experts
//   sigmoid                g_k * s_k * (1 - s_k) at the chosen experts
//   sigmoid, renormalised  q_k * (1 - s_k) * (g_k - sum g q) at the chosen experts
//
// The choice is that of 64-bit arithmetic, ties to the lowest expert, but made in
// 32 bits.  Each lane sorts keys of its experts: the ordered code of the choice
// value with the lane's index of the expert in its lowest bits.  The sorted keys
// lie in shared memory, the lanes' best ones are compared, and the winner's next
// takes its place, top_k + 1 times.  Then the order is proved: each key taken
// has to stand for more than the next one by more than both can be off.  Where
// that fails (some tokens in a thousand, with a bias) the values themselves are
// compared; what is still too close is ordered in 64 bits, a lane for each of those taken,
// and only where something else may come in is the whole row chosen again.
//
// 65536 x 256 f32 logits in 8 groups with a bias, 47 us with the logits in L2 and 48
// without; the bytes take 10.5 (at 6787 GB/s).  It is bound by instructions and their
// latency (570 a token, 58% of the issue slots; the turns of the selection 10 us, the groups 8, sorting 4, the
// proof 2 to 4), the row is read once.  65536 x 128 bf16 without a bias: 13.6 us.
#include <cfloat>

#include "rows.cuh"

namespace gbs {
namespace {

constexpr int ROUTE_THREADS = 128;
// From so many tokens on 256 experts are 16 lanes' instead of 32 (65536 tokens by
// groups 52 us instead of 58, 8192 about the same, 64 4.6 instead of 3.5).
constexpr uint32_t MANY_TOKENS = 4096;
constexpr float U = 5.9604644775390625e-8f;  // 2^-24, the relative error of a rounding
constexpr uint32_t FULL = 0xFFFFFFFFu;

struct RouteParams {
    const void *logits;
    size_t stride;
    uint32_t tokens, experts, top_k;
    const float *bias;  // nullptr: none
    int sigmoid, renorm;
    float scale;
    uint32_t groups, each, top_groups, group_top;
    uint32_t span;  // lanes of a group where that is a power of two, else 0
    int vec, bias_vec;  // rows (the bias) as words of 16 bytes
    void *ids;
    int id_bytes;
    void *weights;  // route: out; grad: the weights' gradient
    int weight_type;
    void *d_logits;  // grad only
    size_t d_stride;
    int d_vec;
    uint32_t chosen_bytes, token_bytes;  // of a token's part of shared memory: entries of the choice; all
};

// Sums and maxima over the L lanes that share a token.
template <int L> __device__ __forceinline__ uint32_t max_of(uint32_t x) {
    if constexpr (L == 32) {
        return __reduce_max_sync(FULL, x);
    } else {
#pragma unroll
        for (int d = L / 2; d > 0; d /= 2) x = max(x, __shfl_xor_sync(FULL, x, d));
        return x;
    }
}
template <int L> __device__ __forceinline__ float max_of(float x) {
#pragma unroll
    for (int d = L / 2; d > 0; d /= 2) x = fmaxf(x, __shfl_xor_sync(FULL, x, d));
    return x;
}
template <int L, typename F> __device__ __forceinline__ F sum_of(F x) {
#pragma unroll
    for (int d = L / 2; d > 0; d /= 2) x += __shfl_xor_sync(FULL, x, d);
    return x;
}
template <int L> __device__ __forceinline__ uint32_t or_of(uint32_t x) {
#pragma unroll
    for (int d = L / 2; d > 0; d /= 2) x |= __shfl_xor_sync(FULL, x, d);
    return x;
}
template <int L> __device__ __forceinline__ double max_of(double x) {
#pragma unroll
    for (int d = L / 2; d > 0; d /= 2) x = fmax(x, __shfl_xor_sync(FULL, x, d));
    return x;
}

// Ordered codes: larger is better, 0 is no candidate (minus infinity), any NaN
// is above all, and the two zeros are equal.
__device__ __forceinline__ uint32_t code_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);
    const uint32_t c = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
    return x != x ? FULL : x == -INFINITY ? 0u : c;
}
__device__ __forceinline__ float value_of(uint32_t code) {
    return __uint_as_float(code ^ ((uint32_t)(~((int32_t)code >> 31)) | 0x80000000u));
}
__device__ __forceinline__ uint64_t code_of(double x) {
    const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
    const uint64_t c = u ^ ((uint64_t)((int64_t)u >> 63) | 0x8000000000000000ull);
    return x != x ? ~0ull : x == -INFINITY ? 0ull : c;
}

// sigmoid(x), off by at most 10 U of itself (two units of expf and of the
// quotient, the sum and the product), and in 64 bits.
__device__ __forceinline__ float sigmoid_of(float x) {
    const float t = expf(-fabsf(x)), r = __fdividef(1.0f, 1.0f + t);
    return x >= 0.0f ? r : t * r;
}
__device__ __forceinline__ double sigmoid_of(double x) {
    const double t = exp(-fabs(x));
    return (x >= 0.0 ? 1.0 : t) / (1.0 + t);
}

// 2^x and 1 / x by the fast instructions: off by 4 and 2 U.
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float inverse_fast(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float LOG2E = 1.44269502162933349609375f;

// A sorting network (Batcher's odd-even merge), largest first.
__device__ __forceinline__ void order2(uint32_t &a, uint32_t &b) {
    const uint32_t x = max(a, b);
    b = min(a, b);
    a = x;
}
template <int LO, int N, int R> __device__ __forceinline__ void merge_keys(uint32_t *k) {
    if constexpr (2 * R < N) {
        merge_keys<LO, N, 2 * R>(k);
        merge_keys<LO + R, N, 2 * R>(k);
#pragma unroll
        for (int i = LO + R; i + R < LO + N; i += 2 * R) order2(k[i], k[i + R]);
    } else {
        order2(k[LO], k[LO + R]);
    }
}
template <int LO, int N> __device__ __forceinline__ void sort_keys(uint32_t *k) {
    if constexpr (N > 1) {
        sort_keys<LO, N / 2>(k);
        sort_keys<LO + N / 2, N / 2>(k);
        merge_keys<LO, N, 1>(k);
    }
}

// The pack at p, 8 or 16 bytes.
template <typename T, int N> __device__ __forceinline__ Pack<T, N> load_whole(const T *p) {
    Pack<T, N> x;
    uint32_t *w = reinterpret_cast<uint32_t *>(&x);
    if constexpr (N * sizeof(T) == 16) asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(p));
    else asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
    return x;
}

// A lane's V values of a row from e0 on, `fill` past its end.
template <typename T, int V> __device__ __forceinline__ void load_values(float (&x)[V], const T *row, uint32_t e0, uint32_t count, bool vec, float fill) {
    constexpr int N = 16 / (int)sizeof(T) < V ? 16 / (int)sizeof(T) : V;
    if (vec && e0 + V <= count) {
#pragma unroll
        for (int i = 0; i < V; i += N) {
            const Pack<T, N> a = load_whole<T, N>(row + e0 + i);
#pragma unroll
            for (int j = 0; j < N; ++j) x[i + j] = to_f32(a.v[j]);
        }
    } else if (vec) {
#pragma unroll
        for (int i = 0; i < V; i += N) {
            const bool on = e0 + i < count;
            const Pack<T, N> a = load_pack_if<T, N>(row + e0 + i, on);
#pragma unroll
            for (int j = 0; j < N; ++j) x[i + j] = on ? to_f32(a.v[j]) : fill;
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) x[j] = e0 + j < count ? to_f32(row[e0 + j]) : fill;
    }
}

// Keys below this are no candidates: minus infinity's, and 0.
constexpr uint32_t LEAST_KEY = 0x00800000u, INFINITE_KEY = 0xFF800000u;  // the latter: infinity, and NaN above

// A token's choice, in shared memory.
struct Chosen {
    int32_t id;    // -1: none
    uint32_t key;  // its key, then its choice value
};

// What softmax needs of a row: e^(x - top) * inv.
struct Norm {
    float top, inv;
};
template <int L, int V> __device__ __forceinline__ Norm norm_of(const float (&x)[V]) {
    float m = x[0];
#pragma unroll
    for (int j = 1; j < V; ++j) m = fmaxf(m, x[j]);
    m = max_of<L>(m);
    if (m == -INFINITY) m = 0.0f;  // no expert at all: every score is 0
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) s += exp2_fast((x[j] - m) * LOG2E);
    s = sum_of<L>(s);
    return {m, s == 0.0f ? 0.0f : __fdividef(1.0f, s)};
}

// How far a choice value c may be off: U * ((rounds + 1) * largest + |c|), with
// the largest score of the row (softmax: norm.inv, the score at the top; sigmoid:
// 1).  Softmax, in units of U and of that score: 2^x is off by 4, and by 2.25 times
// the distance from the top d for its exponent (the difference's and the product's
// rounding, and the constant's own 0.23); d * e^-d is at most 1 / e.  In the sum the
// same, where d is at most 4.5 on average (1023 others at one distance), and V + 4
// additions; the inverse is off by 4, the product by 1.  Together V + 28, and what
// is of second order.  Sigmoid: 2^x 4 and 1.25 times |x|, which times the score's
// slope is less than 0.4, the sum and inverse 3; the exact functions of the second
// look (expf, a quotient) are off by less.
template <int V> __device__ __forceinline__ constexpr float score_rounds(bool sigmoid) { return sigmoid ? 12.0f : (float)(V + 32); }
constexpr float WIDER = 1.0001f;  // for the roundings of a bound itself

// What a group's two best are worth.  Values next to the type's lowest add up to
// less than 32 bits hold; that is not minus infinity, no candidate, and is held at
// the lowest (far as that is, the order among such groups is then settled in 64 bits).
__device__ __forceinline__ float sum_of_two(float a, float b) { return fmaxf(a + b, -FLT_MAX); }

// Which groups are kept, as bits; worth[] has the groups' order codes.  A
// group without a candidate (code 0) never is.
template <int L, typename C> __device__ __forceinline__ uint32_t keep_groups(const C *worth, uint32_t groups, uint32_t top_groups, uint32_t sub) {
    uint32_t kept = 0;
    for (uint32_t g = sub; g < groups; g += L) {
        const C mine = worth[g];
        uint32_t above = 0;
        for (uint32_t i = 0; i < groups; ++i) above += worth[i] > mine || (worth[i] == mine && i < g);
        if (above < top_groups && mine != 0) kept |= 1u << g;
    }
    return or_of<L>(kept);
}

// The choice in 64 bits: a warp's work, for all of its tokens.  room: the
// token's part of shared memory for L * V codes and the groups' worths.
template <typename T, int L, int V> __device__ __noinline__ void choose_exactly(const RouteParams &p, const T *row, uint32_t experts, uint32_t sub, Chosen *chosen, uint64_t *room) {
    const uint32_t e0 = sub * V;
    const bool sums = p.groups > 1 && p.group_top > 1, scored = p.bias != nullptr || sums;
    double top = 0.0, total = 1.0;
    if (scored && !p.sigmoid) {
        top = -INFINITY;
        for (int j = 0; j < V; ++j)
            if (e0 + j < experts) top = fmax(top, (double)to_f32(row[e0 + j]));
        top = max_of<L>(top);
        if (top == -INFINITY) top = 0.0;
        total = 0.0;
        for (int j = 0; j < V; ++j)
            if (e0 + j < experts) total += exp((double)to_f32(row[e0 + j]) - top);
        total = sum_of<L>(total);
    }
    // the choice values, by which the groups' worths are made
    double *values = reinterpret_cast<double *>(room);
#pragma unroll 4
    for (int j = 0; j < V; ++j) {
        const bool here = e0 + j < experts;
        const double x = here ? (double)to_f32(row[e0 + j]) : -INFINITY;
        double c = x;
        if (scored) {  // no branch between the values' long chains
            c = p.sigmoid ? sigmoid_of(x) : exp(x - top) / total;
            c = x == -INFINITY ? x : c + (here && p.bias ? (double)p.bias[e0 + j] : 0.0);
        }
        values[e0 + j] = c;
    }
    __syncwarp();
    uint32_t kept = FULL;
    uint64_t *worth = room + L * V;
    if (p.groups > 1) {
        for (uint32_t g = sub; g < p.groups; g += L) {
            double a = -INFINITY, b = -INFINITY;
            bool nan = false;
            for (uint32_t i = 0; i < p.each && g * p.each + i < experts; ++i) {
                const double c = values[g * p.each + i];
                nan |= c != c;
                if (c > a) b = a, a = c;
                else if (c > b) b = c;
            }
            const double w = sums && b != -INFINITY ? a + b : a;
            worth[g] = nan ? ~0ull : code_of(w);
        }
        __syncwarp();
        kept = keep_groups<L>(worth, p.groups, p.top_groups, sub);
    }
    uint64_t *code = room;  // in the values' place
    for (int j = 0; j < V; ++j) {
        const uint32_t e = e0 + j;
        double c = values[e];
        if (!p.bias && e < experts) c = (double)to_f32(row[e]);  // without a bias the logits' order
        code[e] = (p.groups > 1 && !((kept >> (e / p.each)) & 1)) || e >= experts ? 0ull : code_of(c);
    }
    uint64_t best = 0;
    uint32_t at = 0;
    auto find = [&]() {
        best = 0;
        for (int j = 0; j < V; ++j)
            if (code[e0 + j] > best) best = code[e0 + j], at = j;
    };
    find();
    const uint32_t lane = threadIdx.x & 31, mine = L == 32 ? FULL : ((1u << (L & 31)) - 1) << (lane & ~(L - 1));
    for (uint32_t s = 0; s < p.top_k; ++s) {
        const uint32_t hi = max_of<L>((uint32_t)(best >> 32)), lo = max_of<L>((uint32_t)(best >> 32) == hi ? (uint32_t)best : 0u);
        const uint64_t m = (uint64_t)hi << 32 | lo;
        const uint32_t b = __ballot_sync(FULL, best == m) & mine;
        if (lane == (uint32_t)__ffs(b) - 1) {
            chosen[s].id = m != 0 ? (int32_t)(e0 + at) : -1;
            if (m != 0) {
                code[e0 + at] = 0;
                find();
            }
        }
    }
    __syncwarp();
}

// Makes sure of a choice that its keys alone do not prove; a warp's work, for all
// of its tokens.  st: what is left of the lane's sorted keys after top_k + 1 were
// taken, L apart and 0 behind the last.  The values themselves are compared first;
// where two of those taken are too close they are ordered in 64 bits, a lane for
// each; and where the groups or something else that is left may come in too, the
// choice is made again.
template <typename T, int L, int V>
__device__ __noinline__ void settle(const RouteParams &p, const T *row, uint32_t experts, uint32_t sub, Chosen *chosen, uint64_t *room, const uint32_t *st, Norm norm,
                                    bool groups_sure, bool on) {
    const bool scored = p.bias != nullptr;
    const float rounds = score_rounds<V>(p.sigmoid);
    // what a key's value is at most, and how far that may be off
    auto at_most = [&](uint32_t key) { return value_of(key | (uint32_t)(V - 1)); };
    auto off_most = [&](uint32_t key) { return scored ? U * ((rounds + 1.0f) * norm.inv + fabsf(at_most(key))) : 0.0f; };
    // choice value and error of an expert; what it is made of
    auto choice = [&](int32_t id, float *x, float *b, float *off) {
        *x = to_f32(row[id]);
        *b = scored ? p.bias[id] : 0.0f;
        if (!scored) {
            *off = 0.0f;
            return *x;
        }
        const float s = p.sigmoid ? sigmoid_of(*x) : expf(*x - norm.top) * norm.inv, c = s + *b;
        *off = U * (rounds * s + norm.inv + fabsf(c));
        return c;
    };
    // the order of those taken, and the least that the last of them may be worth: by keys alone that is any of them
    bool order = true, rest = true;
    float least = INFINITY;
    for (uint32_t s = sub; s < p.top_k; s += L) {
        const Chosen a = chosen[s], n = chosen[s + 1];
        if (a.id < 0) continue;
        float x, b, off, x2, b2, off2;
        const float c = choice(a.id, &x, &b, &off);
        least = c != c ? -INFINITY : fminf(least, __fsub_rd(c, WIDER * off));
        if (n.id < 0) continue;
        const float c2 = choice(n.id, &x2, &b2, &off2);
        if (!(c - c2 > WIDER * (off + off2)) && !(x == x2 && b == b2 && a.id < n.id)) order = false;
    }
    least = -max_of<L>(-least);
    order = or_of<L>(!order) == 0;
    // against all that are left: equals of the last one may be left where that is its place for certain
    if (chosen[p.top_k].id >= 0) {
        const Chosen a = chosen[p.top_k - 1];
        float x, b, off;
        choice(a.id, &x, &b, &off);
        for (; *st >= LEAST_KEY; st += L) {
            if (least - at_most(*st) > WIDER * off_most(*st)) break;  // and all after it
            const int32_t id = (int32_t)(sub * V + V - 1 - (*st & (V - 1)));
            if (!(order && id > a.id && to_f32(row[id]) == x && (scored ? p.bias[id] : 0.0f) == b)) rest = false;
        }
    }
    if (!__any_sync(FULL, on && !(groups_sure && order && rest))) return;
    const bool again = !groups_sure || !rest || p.top_k >= L;
    if (__any_sync(FULL, on && again)) {
        choose_exactly<T, L, V>(p, row, experts, sub, chosen, room);
        return;
    }
    double top = 0.0, total = 1.0;
    if (scored && !p.sigmoid) {
        top = (double)norm.top;
        total = 0.0;
#pragma unroll 4
        for (int j = 0; j < V; ++j) total += exp((sub * V + j < experts ? (double)to_f32(row[sub * V + j]) : -INFINITY) - top);
        total = sum_of<L>(total);
    }
    const int32_t id = sub <= p.top_k ? chosen[sub].id : -1;
    double c = -INFINITY;
    if (id >= 0) {
        c = (double)to_f32(row[id]);
        if (scored) c = (p.sigmoid ? sigmoid_of(c) : exp(c - top) / total) + (double)p.bias[id];
    }
    const uint64_t code = code_of(c);
    uint32_t rank = 0;
    for (uint32_t i = 0; i <= p.top_k; ++i) {
        const uint64_t o = __shfl_sync(FULL, code, i, L);
        const int32_t other = __shfl_sync(FULL, id, i, L);
        rank += o > code || (o == code && (uint32_t)other < (uint32_t)id);
    }
    __syncwarp();
    if (id >= 0) chosen[rank].id = id;
    __syncwarp();
}

// Which groups of p.span lanes are kept, in 64 bits, for sigmoids whose worths are
// too close in 32: the lanes evaluate what is near their group's two best, `least`
// or more, one each at a time.
template <typename T, int L, int V>
__device__ __noinline__ bool keep_span_exactly(const RouteParams &p, const T *row, uint32_t experts, float least, bool sums, uint32_t sub) {
    uint32_t near = 0;
    for (int j = 0; j < V; ++j) {  // the values once more: an array handed over would live in memory
        const uint32_t e = sub * V + j;
        if (e >= experts) break;
        const float x = to_f32(row[e]), c = inverse_fast(1.0f + exp2_fast(x * -LOG2E)) + (p.bias ? p.bias[e] : 0.0f);
        near |= (uint32_t)(c >= least && x != -INFINITY && c != -INFINITY) << j;
    }
    double a = -INFINITY, b = -INFINITY;
    while (__any_sync(FULL, near != 0)) {
        const uint32_t e = sub * V + (near ? __ffs(near) - 1 : 0);
        double v = -INFINITY;
        if (near) v = sigmoid_of((double)to_f32(row[e])) + (p.bias ? (double)p.bias[e] : 0.0);
        b = fmax(b, fmin(a, v));
        a = fmax(a, v);
        near &= near - 1;
    }
    for (uint32_t d = 1; d < p.span; d *= 2) {
        const double o = __shfl_xor_sync(FULL, a, d), u = __shfl_xor_sync(FULL, b, d);
        b = fmax(fmax(b, u), fmin(a, o));
        a = fmax(a, o);
    }
    const uint64_t worth = code_of(sums && b != -INFINITY ? a + b : a);
    const uint32_t lane = threadIdx.x & 31, mine = L == 32 ? FULL : ((1u << (L & 31)) - 1) << (lane & ~(L - 1));
    bool keep = false;
    for (uint32_t g = 0; g < p.top_groups; ++g) {
        const uint64_t own = keep ? 0 : worth;
        const uint32_t hi = max_of<L>((uint32_t)(own >> 32)), lo = max_of<L>((uint32_t)(own >> 32) == hi ? (uint32_t)own : 0u);
        const uint64_t best = (uint64_t)hi << 32 | lo;
        const uint32_t of = __ballot_sync(FULL, !keep && worth == best) & mine;
        if (best != 0 && (((uint32_t)__ffs(of) - 1) ^ lane) < p.span) keep = true;
    }
    return keep;
}

// Whether the lane's group is kept, for groups of p.span lanes: a power of two.
template <typename T, int L, int V>
__device__ __forceinline__ bool keep_span(const RouteParams &p, const T *row, const float (&c)[V], bool sums, bool scored, float largest, uint32_t sub, uint32_t experts,
                                          bool *sure) {
    float a = c[0], b = -INFINITY;
    if (sums) {
#pragma unroll
        for (int j = 1; j < V; ++j) b = fmaxf(b, fminf(a, c[j])), a = fmaxf(a, c[j]);
#pragma unroll
        for (int d = 1; d < L; d *= 2) {
            if ((uint32_t)d >= p.span) break;
            const float o = __shfl_xor_sync(FULL, a, d), u = __shfl_xor_sync(FULL, b, d);
            b = fmaxf(fmaxf(b, u), fminf(a, o));
            a = fmaxf(a, o);
        }
    } else {
#pragma unroll
        for (int j = 1; j < V; ++j) a = fmaxf(a, c[j]);
#pragma unroll
        for (int d = 1; d < L; d *= 2) {
            if ((uint32_t)d >= p.span) break;
            a = fmaxf(a, __shfl_xor_sync(FULL, a, d));
        }
    }
    const bool two = sums && b != -INFINITY;
    const uint32_t worth = code_of(two ? sum_of_two(a, b) : a);  // of all lanes of a group
    // better groups, and equal ones before this; every lane of a group has its worth
    const uint32_t lane = threadIdx.x & 31, self = (lane & (L - 1)) / p.span;
    uint32_t better = 0;
#pragma unroll 8
    for (uint32_t g = 0; g < p.groups; ++g) {
        const uint32_t o = __shfl_sync(FULL, worth, g * p.span, L);
        better += o > worth || (o == worth && g < self);
    }
    bool keep = better < p.top_groups && worth != 0;
    if (scored && p.top_groups < p.groups) {
        // the worst that is kept against the best that is not, by more than the values and their sums may be off
        const uint32_t mine = L == 32 ? FULL : ((1u << (L & 31)) - 1) << (lane & ~(L - 1));
        const uint32_t last = __ballot_sync(FULL, better + 1 == p.top_groups) & mine, next = __ballot_sync(FULL, better == p.top_groups) & mine;
        // (the places differ, so that both are there)
        const uint32_t least = __shfl_sync(FULL, worth, last ? __ffs(last) - 1 : lane), most = __shfl_sync(FULL, worth, next ? __ffs(next) - 1 : lane);
        const uint32_t far = max_of<L>(worth == 0 ? 0u : __float_as_uint(fabsf(a) + (two ? fabsf(b) : 0.0f)));
        const float off = 4.0f * WIDER * U * ((score_rounds<V>(p.sigmoid) + 1.0f) * largest + __uint_as_float(far));
        const bool close = most != 0 && !(value_of(least) - value_of(most) > off);
        if (__any_sync(FULL, close)) {
            if (p.sigmoid) keep = keep_span_exactly<T, L, V>(p, row, experts, (two ? b : a) - off, sums, sub);
            else if (close) *sure = false;
        }
    }
    return keep;
}

// The groups that are kept, as bits, for any groups: by way of shared memory.
template <int L, int V>
__device__ __forceinline__ uint32_t keep_anywhere(const RouteParams &p, const float (&c)[V], bool sums, bool scored, float largest, uint32_t e0, uint32_t sub, uint32_t experts,
                                                  uint64_t *room, bool *sure) {
    float *values = reinterpret_cast<float *>(room);
#pragma unroll
    for (int j = 0; j < V; ++j) values[e0 + j] = c[j];
    __syncwarp();
    uint32_t *worth = reinterpret_cast<uint32_t *>(room + L * V);
    float *off = reinterpret_cast<float *>(worth + p.groups);  // how far a worth may be off
    uint32_t parts = 1;  // lanes that share a group
    while (2 * parts * p.groups <= (uint32_t)L) parts *= 2;
    for (uint32_t g0 = 0; g0 < p.groups; g0 += L / parts) {
        const uint32_t g = g0 + sub / parts, part = sub & (parts - 1);
        float a = -INFINITY, b = -INFINITY;
        bool nan = false;
        for (uint32_t i = part; g < p.groups && i < p.each && g * p.each + i < experts; i += parts) {
            const float v = values[g * p.each + i];
            nan |= v != v;
            b = fmaxf(b, fminf(a, v));
            a = fmaxf(a, v);
        }
        uint32_t some = nan;
        for (uint32_t d = 1; d < parts; d *= 2) {
            const float o = __shfl_xor_sync(FULL, a, d), u = __shfl_xor_sync(FULL, b, d);
            some |= __shfl_xor_sync(FULL, some, d);
            b = fmaxf(fmaxf(b, u), fminf(a, o));
            a = fmaxf(a, o);
        }
        if (part == 0 && g < p.groups) {
            const bool two = sums && b != -INFINITY;
            worth[g] = some ? FULL : code_of(two ? sum_of_two(a, b) : a);
            // each value's error, and the sum's
            off[g] = 2.0f * WIDER * U * ((score_rounds<V>(p.sigmoid) + 1.0f) * largest + fabsf(a) + (two ? fabsf(b) : 0.0f));
        }
    }
    __syncwarp();
    const uint32_t kept = keep_groups<L>(worth, p.groups, p.top_groups, sub);
    if (scored && p.top_groups < p.groups) {
        float least = INFINITY, most = -INFINITY;  // the worst that is kept, the best that is not
        for (uint32_t g = sub; g < p.groups; g += L) {
            if (worth[g] == FULL) *sure = false;
            else if ((kept >> g) & 1) least = fminf(least, value_of(worth[g]) - off[g]);
            else if (worth[g] != 0) most = fmaxf(most, value_of(worth[g]) + off[g]);
        }
        least = -max_of<L>(-least);
        most = max_of<L>(most);
        if (!(least > most)) *sure = false;
    }
    return kept;
}

// A token is L lanes' work, V experts each; a warp has 32 / L tokens.
template <typename T, int L, int V> __global__ void __launch_bounds__(ROUTE_THREADS) route_kernel(const __grid_constant__ RouteParams p) {
    extern __shared__ __align__(16) unsigned char shared[];
    wait_for_earlier();
    const uint32_t lane = threadIdx.x & 31, sub = lane & (L - 1), here = threadIdx.x / L;
    const uint32_t t = blockIdx.x * (ROUTE_THREADS / L) + here;
    const bool on = t < p.tokens;
    const uint32_t experts = on ? p.experts : 0, e0 = sub * V;
    const T *row = static_cast<const T *>(p.logits) + (on ? (size_t)t * p.stride : 0);
    Chosen *chosen = reinterpret_cast<Chosen *>(shared + here * p.token_bytes);
    uint64_t *room = reinterpret_cast<uint64_t *>(shared + here * p.token_bytes + p.chosen_bytes);
    const bool sums = p.groups > 1 && p.group_top > 1, scored = p.bias != nullptr || sums;

    float x[V];
    load_values<T, V>(x, row, e0, experts, p.vec, -INFINITY);
    Norm norm = {0.0f, 1.0f};
    if (!p.sigmoid && (scored || !p.renorm)) norm = norm_of<L, V>(x);
    bool sure = true, open = true;  // whether the lane's group can be chosen from, with spans
    uint32_t keys[V];
    {
        float c[V];
#pragma unroll
        for (int j = 0; j < V; ++j) c[j] = x[j];
        if (scored) {
            float b[V];
#pragma unroll
            for (int j = 0; j < V; ++j) b[j] = 0.0f;
            if (p.bias) load_values<float, V>(b, p.bias, e0, experts, p.bias_vec, 0.0f);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float s = p.sigmoid ? inverse_fast(1.0f + exp2_fast(x[j] * -LOG2E)) : exp2_fast((x[j] - norm.top) * LOG2E) * norm.inv;
                c[j] = x[j] == -INFINITY ? -INFINITY : s + b[j];
            }
        }
        uint32_t kept = FULL;
        if (p.groups > 1) {
            if (p.span) open = keep_span<T, L, V>(p, row, c, sums, scored, norm.inv, sub, experts, &sure);
            else kept = keep_anywhere<L, V>(p, c, sums, scored, norm.inv, e0, sub, experts, room, &sure);
        }
        if (p.bias == nullptr)
#pragma unroll
            for (int j = 0; j < V; ++j) c[j] = x[j] + 0.0f;  // one zero, one NaN
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const uint32_t u = __float_as_uint(c[j]), k = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
            keys[j] = (k & ~(uint32_t)(V - 1)) | (uint32_t)(V - 1 - j);
        }
        if (kept != FULL) {
            uint32_t g = e0 / p.each, r = e0 % p.each;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (!((kept >> (g & 31)) & 1)) keys[j] = 0;
                if (++r == p.each) r = 0, ++g;
            }
        }
    }
    sort_keys<0, V>(keys);
    if (p.groups > 1 && keys[0] >= INFINITE_KEY) sure = false;  // NaN has no place in the groups' sums
    uint32_t *keys_left = reinterpret_cast<uint32_t *>(room) + sub;
    for (uint32_t s = sub; s <= p.top_k; s += L) chosen[s] = {-1, 0};
    __syncwarp();
#pragma unroll
    for (int j = 0; j < V; ++j) keys_left[j * L] = keys[j];
    keys_left[V * L] = 0;
    uint32_t head = open ? keys[0] : 0u, left = smem_u32(keys_left) + (open ? 0 : V * L * 4), to = smem_u32(chosen);
    // 16-bit logits have bits to spare for the index: their order is exact
    const bool exact = sizeof(T) == 2 && p.bias == nullptr;
    const uint32_t lower = (L == 32 ? FULL : ((1u << (L & 31)) - 1) << (lane & ~(L - 1))) & lanemask_lt();
#pragma unroll 3
    for (uint32_t s = p.top_k + (exact ? 0 : 1); s > 0; --s, to += sizeof(Chosen)) {
        const uint32_t m = max(max_of<L>(head), LEAST_KEY);
        const bool hit = (head ^ m) < (uint32_t)V;  // the lowest lane of equals has the lowest expert
        const uint32_t b = __ballot_sync(FULL, hit);
        // the lane's best goes to the choice, its next takes its place
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\t@q st.shared.v2.u32 [%3], {%4, %0};\n\t@q add.u32 %1, %1, %5;\n\t"
                     "@q ld.shared.u32 %0, [%1];\n\t}"
                     : "+r"(head), "+r"(left)
                     : "r"((uint32_t)(hit && (b & lower) == 0)), "r"(to), "r"(e0 + V - 1 - (head & (V - 1))), "n"(4 * L)
                     : "memory");
    }
    const uint32_t *st = keys_left + (left - smem_u32(keys_left)) / 4;
    __syncwarp();
    bool plain = true;
    if (!exact) {
        // by the keys: the least that one stands for against the most of the next one's
        const float off = p.bias ? 2.0f * (score_rounds<V>(p.sigmoid) + 1.0f) * norm.inv : 0.0f, of = p.bias ? 1.0f : 0.0f;
        for (uint32_t s = sub; s < p.top_k; s += L) {
            const uint32_t a = chosen[s].key, n = chosen[s + 1].key;
            const float low = value_of(a & ~(uint32_t)(V - 1)), high = value_of(n | (uint32_t)(V - 1));
            if (n >= LEAST_KEY && !(low - high > WIDER * U * (off + of * (fabsf(low) + fabsf(high))))) plain = false;
        }
    }
    // every lane takes part, whatever its own say
    if (__any_sync(FULL, !plain || !sure)) {
        if (exact) choose_exactly<T, L, V>(p, row, experts, sub, chosen, room);
        else settle<T, L, V>(p, row, experts, sub, chosen, room, st, norm, sure, on);
    }

    auto store = [&](uint32_t s, int32_t id, float w) {
        const size_t at = (size_t)t * p.top_k + s;
        if (p.id_bytes == 8) static_cast<int64_t *>(p.ids)[at] = id;
        else static_cast<int32_t *>(p.ids)[at] = id;
        if (p.weight_type == ROW_F32) static_cast<float *>(p.weights)[at] = w;
        else static_cast<T *>(p.weights)[at] = from_f32<T>(w);
    };
    // the chosen experts' weights, a lane for each slot
    bool small = false;
    if (p.top_k <= L) {
        const int32_t id = on && sub < p.top_k ? chosen[sub].id : -1;
        float w = id >= 0 ? to_f32(row[id]) : -INFINITY;
        // without a bias the first one's logit is the largest
        float top = norm.top;
        if (p.renorm && !scored) top = __shfl_sync(FULL, w, 0, L);
        w = id < 0 ? 0.0f : p.sigmoid ? sigmoid_of(w) : expf(w - top);
        float by = norm.inv;
        if (p.renorm) {
            const float sum = sum_of<L>(w);
            small = __any_sync(FULL, id >= 0 && !(sum > 6e-8f));  // so that a denormal's rounding stays one
            // a row whose softmax is NaN, by which the choice was made, has no other weights
            by = __fdividef(1.0f, sum) + 0.0f * norm.inv;
        }
        if (!small) {
            if (id >= 0) w *= by * p.scale;
            if (on && sub < p.top_k) store(sub, id, w);
            return;
        }
    }
    // more slots than lanes, or scores that are all small: divided by the largest chosen one's exponential
    float top = -INFINITY;
    if (p.renorm) {
        for (uint32_t s = sub; s < p.top_k; s += L)
            if (on && chosen[s].id >= 0) top = fmaxf(top, to_f32(row[chosen[s].id]));
        top = max_of<L>(top);
        if (top == -INFINITY) top = 0.0f;
        if (p.sigmoid) top = fminf(top, 0.0f);
    }
    auto score = [&](int32_t id) {
        const float v = to_f32(row[id]);
        if (!p.renorm) return p.sigmoid ? sigmoid_of(v) : expf(v - norm.top) * norm.inv;
        return p.sigmoid ? __fdividef(expf(fminf(v, 0.0f) - top), 1.0f + expf(-fabsf(v))) : expf(v - top);
    };
    float sum = 0.0f;
    if (p.renorm) {
        for (uint32_t s = sub; s < p.top_k; s += L)
            if (on && chosen[s].id >= 0) sum += score(chosen[s].id);
        sum = sum_of<L>(sum) + 0.0f * norm.inv;
    }
    if (!on) return;
    for (uint32_t s = sub; s < p.top_k; s += L) {
        const int32_t id = chosen[s].id;
        float w = id >= 0 ? score(id) : 0.0f;
        if (p.renorm && id >= 0) w = w / sum;
        store(s, id, w * p.scale);
    }
}

// The gradient where a token has more slots than lanes: its slots add to the row
// in shared memory one after the other.  Bound by that order and the slots' loads, not
// by bytes: 65536 x 8 with two choices 4.0 to 4.6 us (0.4 to 0.8 of bytes; about 3.8 is
// what calls in a row cost), with four 4.6 to 5.8; 16384 x 256 f32 with 40 choices 18 to
// 22 (3.6 to 5.7).
template <typename T, int L, int V> __global__ void __launch_bounds__(ROUTE_THREADS) route_grad_kernel(const __grid_constant__ RouteParams p) {
    extern __shared__ __align__(16) unsigned char shared[];
    wait_for_earlier();
    const uint32_t lane = threadIdx.x & 31, sub = lane & (L - 1), here = threadIdx.x / L;
    const uint32_t t = blockIdx.x * (ROUTE_THREADS / L) + here;
    const bool on = t < p.tokens;
    const uint32_t experts = on ? p.experts : 0, e0 = sub * V;
    const T *row = static_cast<const T *>(p.logits) + (on ? (size_t)t * p.stride : 0);
    float *d = reinterpret_cast<float *>(shared + here * p.token_bytes);  // L * V values
#pragma unroll
    for (int j = 0; j < V; ++j) d[e0 + j] = 0.0f;
    __syncwarp();
    const bool whole = !p.sigmoid && !p.renorm;  // every logit has a gradient
    float x[V];
    Norm norm = {0.0f, 1.0f};
    if (whole) {
        load_values<T, V>(x, row, e0, experts, p.vec, -INFINITY);
        norm = norm_of<L, V>(x);
    }
    auto id_at = [&](uint32_t s) {
        const size_t at = (size_t)t * p.top_k + s;
        const int64_t id = p.id_bytes == 8 ? static_cast<const int64_t *>(p.ids)[at] : static_cast<const int32_t *>(p.ids)[at];
        return id >= 0 && id < (int64_t)experts ? (int32_t)id : -1;
    };
    auto g_at = [&](uint32_t s) {
        const size_t at = (size_t)t * p.top_k + s;
        return p.scale * (p.weight_type == ROW_F32 ? static_cast<const float *>(p.weights)[at] : to_f32(static_cast<const T *>(p.weights)[at]));
    };
    float top = 0.0f;
    if (p.renorm) {
        top = -INFINITY;
        for (uint32_t s = sub; on && s < p.top_k; s += L) {
            const int32_t id = id_at(s);
            if (id >= 0) top = fmaxf(top, to_f32(row[id]));
        }
        top = max_of<L>(top);
        if (top == -INFINITY) top = 0.0f;
        if (p.sigmoid) top = fminf(top, 0.0f);
    }
    auto score = [&](float v) {
        if (!p.renorm) return p.sigmoid ? sigmoid_of(v) : expf(v - norm.top) * norm.inv;
        return p.sigmoid ? __fdividef(expf(fminf(v, 0.0f) - top), 1.0f + expf(-fabsf(v))) : expf(v - top);
    };
    float sum = 0.0f, dot = 0.0f;
    if (p.renorm || whole) {
        for (uint32_t s = sub; on && s < p.top_k; s += L) {
            const int32_t id = id_at(s);
            if (id < 0) continue;
            const float v = score(to_f32(row[id]));
            sum += v;
            dot += v * g_at(s);
        }
        sum = sum_of<L>(sum);
        dot = sum_of<L>(dot);
    }
    const float inv = p.renorm && sum != 0.0f ? 1.0f / sum : p.renorm ? 0.0f : 1.0f;
    // the same expert twice counts twice: one slot of a token after the other
    for (uint32_t s = 0; s < p.top_k; s += L) {
        int32_t id = -1;
        float v = 0.0f;
        if (on && s + sub < p.top_k) id = id_at(s + sub);
        if (id >= 0) {
            const float g = g_at(s + sub), l = to_f32(row[id]);
            if (whole) v = g;
            else if (!p.renorm) v = g * sigmoid_of(l) * sigmoid_of(-l);
            else v = score(l) * inv * (g - dot * inv) * (p.sigmoid ? sigmoid_of(-l) : 1.0f);
        }
        for (uint32_t i = 0; i < L && s + i < p.top_k; ++i) {
            if (sub == i && id >= 0) d[id] += v;
            __syncwarp();
        }
    }
    if (!on) return;
    T *out = static_cast<T *>(p.d_logits) + (size_t)t * p.d_stride;
    float r[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        r[j] = d[e0 + j];
        if (whole) r[j] = expf(x[j] - norm.top) * norm.inv * (r[j] - dot);
    }
    if (p.d_vec) {
        constexpr int N = 16 / (int)sizeof(T) < V ? 16 / (int)sizeof(T) : V;
#pragma unroll
        for (int i = 0; i < V; i += N) {
            Pack<T, N> a;
#pragma unroll
            for (int j = 0; j < N; ++j) a.v[j] = from_f32<T>(r[i + j]);
            if (e0 + i < experts) store_pack(out + e0 + i, a);
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (e0 + j < experts) out[e0 + j] = from_f32<T>(r[j]);
    }
}

// The gradient where a token's slots have a lane each.  The row is written as if
// nothing were chosen, then the chosen experts' lanes write theirs over it.  Lanes
// hold every L-th pack of a row.  Near its bytes: 65536 x 128 f32 softmax 13.4 us
// with other inputs each time, 10.6 with the logits in L2 (71 MB read and written, 10.5
// at 6787 GB/s), 16384 x 256 sigmoid 5.5 us (18.9 MB written, in one wave of CTAs).  By
// way of shared memory, with the logits in L2, it took 25.6 and 13.5.
template <typename T, int L, int V> __global__ void __launch_bounds__(ROUTE_THREADS) route_grad_slots_kernel(const __grid_constant__ RouteParams p) {
    extern __shared__ __align__(16) unsigned char shared[];
    constexpr int N = 16 / (int)sizeof(T) < V ? 16 / (int)sizeof(T) : V;
    wait_for_earlier();
    const uint32_t lane = threadIdx.x & 31, sub = lane & (L - 1), here = threadIdx.x / L;
    const uint32_t t = blockIdx.x * (ROUTE_THREADS / L) + here;
    const bool on = t < p.tokens;
    const uint32_t experts = on ? p.experts : 0;
    const T *row = static_cast<const T *>(p.logits) + (on ? (size_t)t * p.stride : 0);
    T *out = static_cast<T *>(p.d_logits) + (on ? (size_t)t * p.d_stride : 0);
    uint32_t *tag = reinterpret_cast<uint32_t *>(shared + here * p.token_bytes);  // [experts]
    const bool whole = !p.sigmoid && !p.renorm, packs = p.vec && p.d_vec;

    int32_t id = -1;
    float g = 0.0f, l = -INFINITY;
    if (on && sub < p.top_k) {
        const size_t at = (size_t)t * p.top_k + sub;
        const int64_t named = p.id_bytes == 8 ? static_cast<const int64_t *>(p.ids)[at] : static_cast<const int32_t *>(p.ids)[at];
        id = named >= 0 && named < (int64_t)experts ? (int32_t)named : -1;
        g = p.scale * (p.weight_type == ROW_F32 ? static_cast<const float *>(p.weights)[at] : to_f32(static_cast<const T *>(p.weights)[at]));
    }
    float x[V];
    Norm norm = {0.0f, 1.0f};
    if (whole) {
        if (packs) {
#pragma unroll
            for (int i = 0; i < V; i += N) {
                const uint32_t e = ((i / N) * L + sub) * N;
                const Pack<T, N> a = load_pack_if<T, N>(row + e, e < experts);
#pragma unroll
                for (int j = 0; j < N; ++j) x[i + j] = e < experts ? to_f32(a.v[j]) : -INFINITY;
            }
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) x[j] = j * L + sub < experts ? to_f32(row[j * L + sub]) : -INFINITY;
        }
    }
    if (id >= 0) l = to_f32(row[id]), tag[id] = sub;
    if (whole) norm = norm_of<L, V>(x);
    // scores over e^top, the largest chosen one's where they are renormalised
    float top = norm.top;
    if (p.renorm) {
        top = max_of<L>(l);
        if (top == -INFINITY) top = 0.0f;
        if (p.sigmoid) top = fminf(top, 0.0f);
    }
    float v = 0.0f;
    if (id >= 0) {
        if (!p.sigmoid) v = expf(l - top) * norm.inv;
        else v = p.renorm ? __fdividef(expf(fminf(l, 0.0f) - top), 1.0f + expf(-fabsf(l))) : sigmoid_of(l);
    }
    float sum = 0.0f, dot = 0.0f;
    if (p.renorm || whole) {
        dot = sum_of<L>(v * (id >= 0 ? g : 0.0f));
        if (p.renorm) {
            sum = sum_of<L>(v);
            const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
            v *= inv;
            dot *= inv;
        }
    }
    // the same expert twice counts twice: its first slot writes the sum, in the slots' order
    __syncwarp();
    const bool twice = __any_sync(FULL, id >= 0 && tag[id] != sub);
    if (twice) {
        float all = 0.0f;
        uint32_t many = 0;
        bool first = true;
        for (uint32_t i = 0; i < p.top_k; ++i) {
            const int32_t other = __shfl_sync(FULL, id, i, L);
            const float og = __shfl_sync(FULL, g, i, L);
            if (other == id) {
                all += og;
                ++many;
                first = first && i >= sub;
            }
        }
        // v * (g - dot) of every slot, or in the whole row v * (all of their g - dot) once
        g = whole || !p.renorm ? all : all - (float)(many - 1) * dot;
        if (!first) id = -1;
    }
    float d;
    if (whole) d = v * (g - dot);
    else if (!p.renorm) d = g * v * sigmoid_of(-l);
    else d = v * (g - dot) * (p.sigmoid ? sigmoid_of(-l) : 1.0f);
    if (packs) {
#pragma unroll
        for (int i = 0; i < V; i += N) {
            const uint32_t e = ((i / N) * L + sub) * N;
            Pack<T, N> a;
#pragma unroll
            for (int j = 0; j < N; ++j) a.v[j] = from_f32<T>(whole ? exp2_fast((x[i + j] - norm.top) * LOG2E) * norm.inv * -dot : 0.0f);
            if (e < experts) store_pack(out + e, a);
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (j * L + sub < experts) out[j * L + sub] = from_f32<T>(whole ? exp2_fast((x[j] - norm.top) * LOG2E) * norm.inv * -dot : 0.0f);
    }
    __syncwarp();
    if (id >= 0) out[id] = from_f32<T>(d);
}

template <typename T, int L, int V> cudaError_t launch(RouteParams &p, cudaStream_t stream) {
    constexpr uint32_t TOKENS = ROUTE_THREADS / L;
    p.chosen_bytes = (p.top_k + 2) / 2 * 2 * (uint32_t)sizeof(Chosen);
    p.token_bytes = p.chosen_bytes + L * V * 8 + (L * V < 32 ? L * V : 32) * 8;
    const uint32_t span = p.each % V == 0 ? p.each / V : 0;
    p.span = span <= L && (span & (span - 1)) == 0 ? span : 0;
    return launch_next(route_kernel<T, L, V>, dim3((p.tokens + TOKENS - 1) / TOKENS), dim3(ROUTE_THREADS), TOKENS * p.token_bytes, stream, p);
}
template <typename T, int L, int V> cudaError_t launch_grad(RouteParams &p, cudaStream_t stream) {
    constexpr uint32_t TOKENS = ROUTE_THREADS / L;
    p.token_bytes = L * V * 4;
    return launch_next(p.top_k <= L ? route_grad_slots_kernel<T, L, V> : route_grad_kernel<T, L, V>, dim3((p.tokens + TOKENS - 1) / TOKENS),
                       dim3(ROUTE_THREADS), TOKENS * p.token_bytes, stream, p);
}

// Lanes for a token and experts for a lane, by the experts.  More experts a lane
// are fewer instructions a token, and a longer way for one.  65536 tokens, us: 32
// experts by 4 lanes 5.2, by 8 lanes 8.0; 128 bf16 by 8 lanes 14.5, by 16 22.4; 64
// f32 by 8 lanes 11.5, by 4 16.7; 256 by 8 lanes 99 (32 keys a lane leave few
// warps, and few bits for the proof).  The gradient sorts nothing: more lanes.
template <typename T> cudaError_t launch_for(RouteParams &p, bool grad, cudaStream_t stream) {
    if (grad) {
        if (p.experts <= 8) return launch_grad<T, 1, 8>(p, stream);
        if (p.experts <= 32) return launch_grad<T, 8, 4>(p, stream);
        if (p.experts <= 64) return launch_grad<T, 8, 8>(p, stream);
        if (p.experts <= 128) return launch_grad<T, 16, 8>(p, stream);
        if (p.experts <= 256) return launch_grad<T, 32, 8>(p, stream);
        if (p.experts <= 512) return launch_grad<T, 32, 16>(p, stream);
        return launch_grad<T, 32, 32>(p, stream);
    }
    if (p.experts <= 8) return launch<T, 1, 8>(p, stream);
    if (p.experts <= 32) return launch<T, 4, 8>(p, stream);
    if (p.experts <= 64) return launch<T, 8, 8>(p, stream);
    if (p.experts <= 128) return launch<T, 8, 16>(p, stream);
    if (p.experts <= 256) return p.tokens >= MANY_TOKENS ? launch<T, 16, 16>(p, stream) : launch<T, 32, 8>(p, stream);
    if (p.experts <= 512) return launch<T, 32, 16>(p, stream);
    return launch<T, 32, 32>(p, stream);
}

}  // namespace

static cudaError_t route(const RouteJob &job, bool grad, cudaStream_t stream, int *launches) {
    if (job.num_tokens == 0) return cudaSuccess;
    RouteParams p = {};
    p.logits = job.logits.base;
    p.stride = job.logits.stride;
    p.tokens = (uint32_t)job.num_tokens;
    p.experts = job.num_experts;
    p.top_k = job.top_k;
    p.bias = job.bias;
    p.sigmoid = job.sigmoid;
    p.renorm = job.renormalise;
    p.scale = job.scale;
    p.groups = job.num_groups;
    p.each = job.num_groups > 0 ? job.num_experts / job.num_groups : job.num_experts;
    p.top_groups = job.top_groups;
    p.group_top = job.group_top;
    p.vec = whole_packs(&job.logits, 1, job.num_experts);
    const Rows bias = {const_cast<float *>(job.bias), 0, ROW_F32};
    p.bias_vec = whole_packs(&bias, 1, job.num_experts);
    p.ids = job.ids;
    p.id_bytes = job.id_bytes;
    p.weights = job.weights;
    p.weight_type = job.weight_type;
    p.d_logits = job.d_logits.base;
    p.d_stride = job.d_logits.stride;
    p.d_vec = whole_packs(&job.d_logits, 1, job.num_experts);
    const cudaError_t e = job.logits.type == ROW_F32   ? launch_for<float>(p, grad, stream)
                          : job.logits.type == ROW_F16 ? launch_for<__half>(p, grad, stream)
                                                       : launch_for<__nv_bfloat16>(p, grad, stream);
    if (e == cudaSuccess) ++*launches;
    timing_mark(stream);
    return e;
}

cudaError_t launch_route(const RouteJob &job, cudaStream_t stream, int *launches) { return route(job, false, stream, launches); }
cudaError_t launch_route_grad(const RouteJob &job, cudaStream_t stream, int *launches) { return route(job, true, stream, launches); }

}  // namespace gbs

// Verification of drafted tokens against the target's probabilities, from given random numbers.
//
// A walk over a sequence's tree holds the weights w of the node it is at, w_i = exp(x_i - max x) of the scaled logits, and
// their sum z: p = w / z. A draft c is kept if u q(c) z < w_c. One that is not kept leaves w_i = max(w_i / z - q_i, 0), or
// w_c = 0 where drafts come without probabilities, with a new sum. The next token is the first whose running sum of
// w exceeds u z.
//
// A cluster of CTAs walks a sequence, each with its share of the vocabulary's weights in shared memory as fp32, so that a
// row of logits is read once however many children are tried. Each step over the weights ends with one exchange: every
// CTA tells the others its part of the sum and, if it has it, the weight of the draft that is tried next; all of them then
// come to the same decision. Which token is drawn hangs on sums over the whole vocabulary next to a random border, so sums
// are kept as a pair of floats (the rounding of each addition is carried along), 44 bits and more; the weights
// themselves are rounded as fp32 operations round them, one by one.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdio>

#include "wq4_cache.cuh"

namespace wq4 {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBlock = 1024;            // weights whose sums are held while the next token is searched
constexpr int kMaxShare = 50 * 1024;    // weights of a CTA: 200 KB
constexpr int kVerifyMaxV = 400000;

struct VerifyArgs {
    const void* logits;
    const long long* tokens;
    const int *parents, *starts;
    const float *draft_probs, *temperature, *uniforms, *final_uniforms;
    int *accepted, *path;
    long long* next_tokens;
    long long ld, ldp;
    int B, T, max_tokens, V, ld_path;
    int cluster, share;                 // CTAs of a sequence; weights of each, a multiple of kBlock
    unsigned int* status;
};

// A sum and what its additions rounded off (D. E. Knuth, The art of computer programming 2, 4.2.2: the error of
// s = a + b is (a - (s - t)) + (b - t) with t = s - a, exactly).
struct Sum {
    float s, c;
    __device__ __forceinline__ void add(float x) {
        const float t = __fadd_rn(s, x), y = __fsub_rn(t, s);
        c = __fadd_rn(c, __fadd_rn(__fsub_rn(s, __fsub_rn(t, y)), __fsub_rn(x, y)));
        s = t;
    }
    __device__ __forceinline__ void add(const Sum& o) {
        add(o.s);
        c = __fadd_rn(c, o.c);
    }
    __device__ __forceinline__ double value() const { return static_cast<double>(s) + static_cast<double>(c); }
};
__device__ __forceinline__ Sum warp_sum(Sum x) {
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        Sum o;
        o.s = __shfl_xor_sync(0xffffffffu, x.s, d);
        o.c = __shfl_xor_sync(0xffffffffu, x.c, d);
        x.add(o);
    }
    return x;                                        // (lanes may differ in the last bits; lane 0's counts)
}

// What a CTA tells the others at the end of a step.
struct Part {
    float s, c;                         // its sum; or, of a row's first step, its largest logit and (greedy) that one's place
    float w;                            // the weight of the draft that is tried next, -1 where it is another CTA's
    int pad;
};

struct Shared {
    Part part[2][kMaxCluster];          // [turn][CTA]: written by the others
    Sum sum[kWarps];
    float top[kWarps];
    int top_at[kWarps];
    double block[kMaxShare / kBlock];
    int found;
};

__device__ __forceinline__ void st_cluster(uint32_t addr, const Part& p) {
    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(__float_as_uint(p.s)),
                 "r"(__float_as_uint(p.c)), "r"(__float_as_uint(p.w)), "r"(p.pad)
                 : "memory");
}

template <int DT>
__device__ __forceinline__ float logit(const void* p, long long i) {
    if constexpr (DT == WQ4_FP32) return static_cast<const float*>(p)[i];
    else return to_f32<DT == WQ4_BF16>(static_cast<const uint16_t*>(p)[i]);
}

template <int DT>
__global__ void __launch_bounds__(kThreads) verify_kernel(const VerifyArgs a) {
    extern __shared__ float w[];                     // this CTA's weights
    __shared__ Shared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = a.cluster, rank = C > 1 ? static_cast<int>(cluster_rank()) : 0, b = blockIdx.x / C;
    const int v0 = rank * a.share, mine = max(0, min(a.share, a.V - v0));   // vocabulary [v0, v0 + mine)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (C > 1) cluster_sync();                       // (every CTA is there before anything is sent to it)
    int turn = 0;
    // Sends this CTA's part to all, waits for theirs.
    auto exchange = [&](Part p) {
        if (tid < C) {
            if (C > 1) st_cluster(map_to_rank(smem_u32(&sh.part[turn][rank]), tid), p);
            else sh.part[turn][0] = p;
        }
        __syncwarp();
        if (C > 1) cluster_sync();
        else __syncthreads();
        turn ^= 1;                                   // (a CTA may send its next part while another reads these)
        return turn ^ 1;
    };
    // The CTA's sum from every thread's, in all threads.
    auto cta_sum = [&](Sum x) {
        x = warp_sum(x);
        if (lane == 0) sh.sum[warp] = x;
        __syncthreads();
        Sum t{0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kWarps; ++i) t.add(sh.sum[i]);
        __syncthreads();
        return t;
    };
    const int s0 = a.starts[b], s1 = a.starts[b + 1];
    int n = static_cast<int>(static_cast<unsigned>(s1) - static_cast<unsigned>(s0));
    if (s0 < 0 || s1 < s0 || s1 > a.T || n > a.max_tokens) {
        if (tid == 0) atomicOr(a.status, kStatusBadIndex);
        n = 0;
    }
    const float heat = a.temperature ? a.temperature[b] : 1.f;
    const bool greedy = heat == 0.f;
    const float inv_heat = greedy ? 1.f : __frcp_rn(heat);
    bool fine = n > 0 && heat >= 0.f && !isinf(heat);
    int node = 0, kept = 0, j = 0;                   // j: the last draft tried
    double z = 0;
    int* path = a.path + static_cast<long long>(b) * a.ld_path;

    // The next draft to try after j: a child of the node whose token exists.
    long long draft = 0;
    auto next_draft = [&] {
        while (++j < n) {
            if (a.parents[s0 + j] != node) continue;
            draft = a.tokens[s0 + j];
            if (draft >= 0 && draft < a.V) return;
        }
    };
    // Adds up what the CTAs told: z, and the draft's weight.
    float draft_w = 0.f;
    auto take = [&](int was) {
        double s = 0;
        draft_w = -1.f;
        for (int i = 0; i < C; ++i) {
            const Part& p = sh.part[was][i];
            s += static_cast<double>(p.s) + static_cast<double>(p.c);
            draft_w = fmaxf(draft_w, p.w);
        }
        return s;
    };
    auto draft_here = [&] {                          // (after the CTA's weights are written)
        const long long at = draft - v0;
        return j < n && at >= 0 && at < mine ? w[at] : -1.f;
    };

    while (fine) {
        // ---- the node's row
        const long long row = (s0 + node) * a.ld;
        const long long r0 = row + v0;
        float top = -INFINITY;
        int top_at = 0x7fffffff;
        bool odd = false;                            // NaN
        for (int i = tid; i < mine; i += kThreads) {
            float x = logit<DT>(a.logits, r0 + i);
            odd |= x != x;
            if (greedy && x > top) top_at = v0 + i;
            x = __fmul_rn(x, inv_heat);
            w[i] = x;
            top = fmaxf(top, x);
        }
        if (odd) top = INFINITY;
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            const float o = __shfl_xor_sync(0xffffffffu, top, d);
            const int at = __shfl_xor_sync(0xffffffffu, top_at, d);
            if (o > top || (o == top && at < top_at)) top_at = at;
            top = fmaxf(top, o);
        }
        if (lane == 0) sh.top[warp] = top, sh.top_at[warp] = top_at;
        __syncthreads();
        top = sh.top[0], top_at = sh.top_at[0];
        for (int i = 1; i < kWarps; ++i) {
            if (sh.top[i] > top || (sh.top[i] == top && sh.top_at[i] < top_at)) top_at = sh.top_at[i];
            top = fmaxf(top, sh.top[i]);
        }
        int was = exchange(Part{top, __int_as_float(top_at), 0.f, 0});
        top = -INFINITY, top_at = 0x7fffffff;
        for (int i = 0; i < C; ++i) {
            const Part& p = sh.part[was][i];
            if (p.s > top || (p.s == top && __float_as_int(p.c) < top_at)) top_at = __float_as_int(p.c);
            top = fmaxf(top, p.s);
        }
        if (isinf(top)) {                            // (either way; NaN as +inf)
            fine = false;
            break;
        }
        Sum part{0.f, 0.f};
        for (int i = tid; i < mine; i += kThreads) {
            const float e = greedy ? (v0 + i == top_at ? 1.f : 0.f) : expf(__fsub_rn(w[i], top));
            w[i] = e;
            part.add(e);
        }
        next_draft();
        part = cta_sum(part);
        was = exchange(Part{part.s, part.c, draft_here(), 0});
        z = take(was);
        // ---- its children
        bool moved = false;
        while (j < n) {
            const float q = a.draft_probs ? a.draft_probs[(s0 + node) * a.ldp + draft] : 1.f;
            if (static_cast<double>(a.uniforms[s0 + j]) * static_cast<double>(q) * z < static_cast<double>(draft_w)) {
                if (rank == 0 && tid == 0) path[kept] = j;
                ++kept;
                node = j;
                moved = true;
                break;
            }
            // what the draft leaves of the target
            const float inv = static_cast<float>(1.0 / z);
            const float* q_row = a.draft_probs + (s0 + node) * a.ldp + v0;
            Sum left{0.f, 0.f};
            if (a.draft_probs) {
                for (int i = tid; i < mine; i += kThreads) left.add(fmaxf(__fsub_rn(__fmul_rn(w[i], inv), q_row[i]), 0.f));
            } else {
                for (int i = tid; i < mine; i += kThreads) left.add(v0 + i == draft ? 0.f : w[i]);
            }
            left = cta_sum(left);
            const long long tried = draft;
            next_draft();
            // the next draft's weight, should this step's count
            float next_w = -1.f;
            const long long at = draft - v0;
            if (j < n && at >= 0 && at < mine)
                next_w = a.draft_probs ? fmaxf(__fsub_rn(__fmul_rn(w[at], inv), q_row[at]), 0.f) : draft == tried ? 0.f : w[at];
            const float kept_w = draft_here();
            __syncthreads();
            was = exchange(Part{left.s, left.c, next_w, __float_as_int(kept_w)});
            const double z_left = take(was);
            if (z_left > 0) {
                if (a.draft_probs) {
                    for (int i = tid; i < mine; i += kThreads) w[i] = fmaxf(__fsub_rn(__fmul_rn(w[i], inv), q_row[i]), 0.f);
                } else if (tid == 0 && tried >= v0 && tried < v0 + mine) {
                    w[tried - v0] = 0.f;
                }
                z = z_left;
            } else {                                 // nothing is left: the weights stay
                draft_w = -1.f;
                for (int i = 0; i < C; ++i) draft_w = fmaxf(draft_w, __int_as_float(sh.part[was][i].pad));
            }
            __syncthreads();
        }
        if (!moved) break;
        __syncthreads();                             // (the weights are overwritten)
    }
    if (rank == 0) {
        for (int i = kept + tid; i < max(1, a.max_tokens - 1); i += kThreads) path[i] = -1;
        if (tid == 0) a.accepted[b] = kept;
    }
    if (!fine) {
        if (rank == 0 && tid == 0) a.next_tokens[b] = -1;
        return;
    }
    // ---- the next token: sums of blocks of 1024 weights, in pieces of 32, each lane's read askew so that the lanes lie in
    // different banks
    auto piece_sum = [&](int block) {
        Sum s{0.f, 0.f};
        const int from = block * kBlock + lane * 32;
        for (int i = 0; i < 32; ++i) {
            const int at = from + ((i + lane) & 31);
            s.add(at < mine ? w[at] : 0.f);
        }
        return s;
    };
    const int blocks = (mine + kBlock - 1) / kBlock;
    for (int k = warp; k < blocks; k += kWarps) {
        const Sum s = warp_sum(piece_sum(k));
        if (lane == 0) sh.block[k] = s.value();
    }
    __syncthreads();
    double here = 0;
    for (int k = 0; k < blocks; ++k) here += sh.block[k];
    const int was = exchange(Part{static_cast<float>(here), static_cast<float>(here - static_cast<double>(static_cast<float>(here))), 0.f, 0});
    double all = 0;
    for (int i = 0; i < C; ++i) all += static_cast<double>(sh.part[was][i].s) + static_cast<double>(sh.part[was][i].c);
    const double aim = static_cast<double>(a.final_uniforms[b]) * all;
    double upto = 0;
    int owner = -1, last = 0;
    for (int i = 0; i < C; ++i) {
        const double s = static_cast<double>(sh.part[was][i].s) + static_cast<double>(sh.part[was][i].c);
        if (s > 0) last = i;
        if (owner < 0 && upto + s > aim) owner = i;
        if (owner < 0) upto += s;
    }
    const bool past = owner < 0;                     // (u z rounded up to all of z): the last token with a weight
    if (past) owner = last;
    if (owner != rank || warp != 0) return;
    int k = -1, last_k = 0;
    for (int i = 0; i < blocks; ++i) {
        const double s = sh.block[i];
        if (s > 0) last_k = i;
        if (k < 0 && !past && upto + s > aim) k = i;
        if (k < 0) upto += s;
    }
    // (where the blocks' sums and the CTA's do not agree to the last bit, the last one with a weight)
    const bool end = k < 0;
    if (end) k = last_k;
    // of the block's 32 pieces, then of the piece's 32 weights, the first whose running sum exceeds the aim
    const double mine_of_32 = piece_sum(k).value();
    auto pick = [&](double x) {                      // the lane
        double run = x;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const double y = __shfl_up_sync(0xffffffffu, run, d);
            if (lane >= d) run += y;
        }
        const unsigned over = __ballot_sync(0xffffffffu, upto + run > aim), some = __ballot_sync(0xffffffffu, x > 0);
        const int at = !end && over ? __ffs(over) - 1 : some ? 31 - __clz(some) : 0;
        if (at > 0) upto += __shfl_sync(0xffffffffu, run, at - 1);
        return at;
    };
    const int piece = pick(mine_of_32);
    const int from = k * kBlock + piece * 32;
    const int at = pick(from + lane < mine ? static_cast<double>(w[from + lane]) : 0.0);
    if (lane == 0) a.next_tokens[b] = v0 + from + at;
}

template <int DT>
int go_verify(const Runtime& rt, const VerifyArgs& a, wq4_stream_t st) {
    auto kern = verify_kernel<DT>;
    static PerDevice ready;
    const int ok = ready.get(rt.device, [&]() -> int {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxShare * 4) == cudaSuccess) return 1;
        cudaGetLastError();
        return -1;
    });
    if (ok <= 0) return WQ4_ERR_CUDA;
    return launch(rt, kern, dim3(static_cast<unsigned>(a.B) * a.cluster), kThreads, a.share * 4, a.cluster, st, a);
}

}  // namespace
}  // namespace wq4

using namespace wq4;

extern "C" int wq4_verify_drafts(const void* logits, long long ld, const long long* tokens, const int* parents, const int* starts,
                                 int B, int T, int max_tokens, int V, int dtype, const float* draft_probs, long long ldp,
                                 const float* temperature, const float* uniforms, const float* final_uniforms, int* accepted,
                                 int* path, int ld_path, long long* next_tokens, wq4_stream_t stream) {
    if (B < 0 || T < 0 || max_tokens < 1 || V < 1 || (dtype != WQ4_BF16 && dtype != WQ4_FP16 && dtype != WQ4_FP32))
        return WQ4_ERR_INVALID;
    if (V > kVerifyMaxV || B > (1 << 27) || max_tokens > (1 << 20)) return WQ4_ERR_UNSUPPORTED;
    if (B == 0) return WQ4_OK;
    if (!starts || !accepted || !path || !next_tokens || !final_uniforms || ld_path < (max_tokens > 1 ? max_tokens - 1 : 1)) return WQ4_ERR_INVALID;
    if (T > 0 && (!logits || !tokens || !parents || !uniforms || ld < V || (draft_probs && ldp < V))) return WQ4_ERR_INVALID;
    if (ld > (1LL << 40) || (draft_probs && ldp > (1LL << 40))) return WQ4_ERR_INVALID;
    if (!aligned_to(logits, dtype == WQ4_FP32 ? 4 : 2) || !aligned_to(tokens, 8) || !aligned_to(next_tokens, 8)) return WQ4_ERR_ALIGN;
    for (const void* p : {static_cast<const void*>(parents), static_cast<const void*>(starts), static_cast<const void*>(draft_probs),
                          static_cast<const void*>(temperature), static_cast<const void*>(uniforms), static_cast<const void*>(final_uniforms),
                          static_cast<const void*>(accepted), static_cast<const void*>(path)})
        if (!aligned_to(p, 4)) return WQ4_ERR_ALIGN;
    Runtime rt;
    if (const int rc = runtime(&rt)) return rc;
    VerifyArgs a{logits, tokens, parents, starts, draft_probs, temperature, uniforms, final_uniforms, accepted, path, next_tokens,
                 ld, ldp, B, T, max_tokens, V, ld_path, 1, 0, rt.status};
    while (a.cluster < kMaxCluster && V > 16 * kBlock * a.cluster) a.cluster *= 2;
    a.share = ((V + a.cluster - 1) / a.cluster + kBlock - 1) / kBlock * kBlock;
    if (rt.trace) std::fprintf(stderr, "wq4: verify_drafts B=%d tokens=%d V=%d cluster=%d\n", B, max_tokens, V, a.cluster);
    if (dtype == WQ4_BF16) return go_verify<WQ4_BF16>(rt, a, stream);
    if (dtype == WQ4_FP16) return go_verify<WQ4_FP16>(rt, a, stream);
    return go_verify<WQ4_FP32>(rt, a, stream);
}

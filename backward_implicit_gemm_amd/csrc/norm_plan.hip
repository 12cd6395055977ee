// norm_plan.hip -- the shapes the resident group-norm kernels take, on the host.
//
// A plan is a vector length N, the vectors a thread holds (NV) and the threads of
// a team (L).  Of the plans that fit, the one of least estimated time is taken:
// a thread's time grows as NV plus a constant for its reductions, and teams past
// what the chip holds at once (4096 waves at these register counts) wait for
// their turn.
#include <algorithm>

#include "gc_norm_res.h"
#include "gc_train.h"
#include "ig_common.h"

namespace gc {
namespace {

constexpr double kWavesAtOnce = 4096;
constexpr int kVectors[] = {1, 2, 3, 4, 8, 16, 32};
constexpr size_t kLdsMost = 64 * 1024;

double cost(double units, int L, int NV, double waste)
{
    return std::max(1.0, units * L / (64 * kWavesAtOnce)) * (2 + NV) * waste;
}

// whether a kernel of L threads that hold NV vectors of N elements each is built
bool holds(bool bwd, int L, int N, int NV)
{
    if (bwd) return N * NV <= kHeldMost && L <= res_threads_bwd(N * NV);
    return NV <= 16 && L <= res_threads_fwd(N * NV);
}

int pow2_at_most(int64_t v)
{
    int p = 1;
    while (int64_t(p) * 2 <= v) p *= 2;
    return p;
}

// Image slots of the backward: each walks B / at_once images, an equal number, and
// enough for its row of partials (8 bytes a channel) to be an eighth of their bytes at
// most (`joined` slots share a row).
int slots_of(const NormGeom &g, int size, double at_once, int joined = 1)
{
    const int fill = (64 + 3 * g.HW * size * joined - 1) / (3 * g.HW * size * joined);
    const int each = std::max(fill, int(g.B / std::max(1.0, at_once)));
    return (g.B + each - 1) / each;
}

bool plan_nchw(const NormGeom &g, int widest, bool bwd, NormResPlan &best)
{
    // the longest vector that lies in one channel, if it has 8 bytes at least; else a
    // full one that straddles
    int N = widest;
    while (N > 1 && g.HW % N) N >>= 1;
    const bool two = N * 2 < widest && g.HW >= widest;
    if (two) N = widest;
    const int64_t M = int64_t(g.Cg) * g.HW, nvec = (M + N - 1) / N;
    double least = 1e300;
    for (int NV : kVectors)
        for (int L = 1; L <= 1024; L *= 2) {
            if (int64_t(L) * NV < nvec || (L > 1 && int64_t(L) * NV >= 4 * nvec)) continue;
            if (NV > 16 || !holds(bwd, L, N, NV)) continue;
            // lanes of several teams read stretches of memory apart from each other
            const double run = double(L) * N * (16 / widest);
            const double c = cost(double(g.B) * g.G, L, NV, NV > 1 && run < 64 ? 64 / run : 1.0);
            if (c >= least) continue;
            NormResPlan q{};
            q.N = N;
            q.NV = NV;
            q.two = two;
            q.L = L;
            q.threads = L > 64 ? L : kResThreads;   // past a wave the workgroup is the team
            q.teams = q.threads / L;
            q.P = pow2_at_most(std::max(1, std::min(64, L / std::max(1, std::min(g.Cg, L)))));
            if (bwd) {
                q.lds_bytes = std::max<size_t>(256, size_t(q.teams) * nvec * 2 * (two ? 2 : 1) * sizeof(float));
                if (q.lds_bytes > kLdsMost) continue;
                q.images = slots_of(g, 16 / widest, kWavesAtOnce * 64 / (double(g.G) * L));
                q.rows = q.images;
                q.grid = (int64_t(q.images) * g.G + q.teams - 1) / q.teams;
            } else {
                q.grid = (int64_t(g.B) * g.G + q.teams - 1) / q.teams;
            }
            if (!launchable(q.grid, q.threads)) continue;
            least = c;
            best = q;
        }
    return least < 1e300;
}

// Small groups whose vectors hold several channels: NCHW planes shorter than a vector,
// or channels last with rows of 1, 2, 4, ... whole vectors a group.
bool plan_small(const NormGeom &g, int widest, bool bwd, NormResPlan &best)
{
    const int N = widest;
    const int64_t M = int64_t(g.Cg) * g.HW;
    int cv = 1;
    if (g.nhwc) {
        cv = g.Cg / N;
        if (bwd || g.Cg % N || cv > 64 || (cv & (cv - 1))) return false;
    } else if (g.HW >= N || M < N) {
        return false;
    }
    const int64_t nvec = (M + N - 1) / N;
    double least = 1e300;
    for (int NV : kVectors)
        for (int L = cv; L <= 64; L *= 2) {
            if (NV > small_vectors(N, g.nhwc) || int64_t(L) * NV < nvec || (L > cv && int64_t(L) * NV >= 4 * nvec)) continue;
            if (g.nhwc && int64_t(L / cv) * NV < g.HW) continue;
            // the stretch of memory a wave reads at once
            const double run = double(g.nhwc ? std::min<int64_t>(g.C, int64_t(64 / L) * g.Cg) : int64_t(L) * N) * (16 / widest);
            if (g.nhwc && run < 64) continue;
            const double c = cost(double(g.B) * g.G, L, NV, NV > 1 && run < 64 ? 64 / run : 1.0);
            if (c >= least) continue;
            NormResPlan q{};
            q.small = 1;
            q.N = N;
            q.NV = NV;
            q.L = L;
            q.threads = kResThreads;
            q.teams = kResThreads / L;
            if (bwd) {
                q.lds_bytes = size_t(q.teams) * M * 2 * sizeof(float);
                if (q.lds_bytes > kLdsMost) continue;
                const int joined = q.teams % g.G == 0 ? q.teams / g.G : 1;
                q.join = joined > 1;
                q.images = slots_of(g, 16 / widest, kWavesAtOnce * 64 / (double(g.G) * L), joined);
                q.grid = (int64_t(q.images) * g.G + q.teams - 1) / q.teams;
                q.rows = q.join ? int(q.grid) : q.images;
            } else {
                q.grid = (int64_t(g.B) * g.G + q.teams - 1) / q.teams;
            }
            if (!launchable(q.grid, q.threads)) continue;
            least = c;
            best = q;
        }
    return least < 1e300;
}

bool plan_nhwc(const NormGeom &g, int widest, int size, bool bwd, NormResPlan &best)
{
    double least = 1e300;
    for (int N = widest; N >= 1; N >>= 1) {
        // slabs of k whole groups, as wide as fits and no narrower than 64 bytes
        const int most = std::max(1, std::min(g.G, 1024 * N / g.Cg));   // a row is 1024 vectors at most
        for (int k = most; k >= 1; --k) {
            if (g.G % k) continue;
            const int CW = k * g.Cg;
            if (k == 1 ? CW < N : CW % N != 0) continue;
            if (k < g.G && CW * size < 64) continue;
            const int CV = (CW + N - 1) / N, slabs = g.G / k;
            const int mix = CW % N ? 2 : g.Cg % N == 0 || k == 1;
            for (int NV : kVectors)
                for (int L = 64; L <= 1024; L *= 2) {
                    if (!holds(bwd, L, N, NV) || CV > L) continue;
                    if (!bwd && !mix && NV > kMixedMost) continue;
                    const int slots = L / CV;
                    if (int64_t(slots) * NV < g.HW) continue;
                    const double c = cost(double(g.B) * slabs, L, NV, CW * size < 128 && k < g.G ? 1.5 : 1.0);
                    if (c >= least) continue;
                    NormResPlan q{};
                    q.N = N;
                    q.NV = NV;
                    q.L = L;
                    q.wave = L == 64;
                    q.threads = q.wave ? kResThreads : L;
                    q.teams = q.threads / L;
                    q.slots = std::min(slots, g.HW);
                    q.CW = CW;
                    q.slabs = slabs;
                    q.Gs = k;
                    q.mix = mix;
                    q.width = mix ? CV : CW;
                    q.fd_cols = make_fastdiv(CV);
                    q.fd_Eg = make_fastdiv(mix ? CV / k : g.Cg);
                    q.P = pow2_at_most(std::max(1, std::min(64, L / k)));
                    q.team_lds = 2 * q.slots * q.width + 2 * k;
                    size_t lds = size_t(q.teams) * q.team_lds * sizeof(float);
                    if (bwd) lds = std::max(lds, size_t(q.teams) * q.slots * CW * 2 * sizeof(float));
                    q.lds_bytes = lds;
                    if (lds > kLdsMost) continue;
                    if (bwd) {
                        const int slots = slots_of(g, size, kWavesAtOnce * 64 / (double(slabs) * L), q.teams);
                        q.rows = (slots + q.teams - 1) / q.teams;
                        q.images = q.rows * q.teams;
                        q.grid = int64_t(q.rows) * slabs;
                    } else {
                        q.grid = (int64_t(g.B) * slabs + q.teams - 1) / q.teams;
                    }
                    if (!launchable(q.grid, q.threads)) continue;
                    least = c;
                    best = q;
                }
        }
        if (least < 1e300) return true;             // shorter vectors only where longer ones fit nowhere
    }
    return false;
}

}  // namespace

namespace {
bool search(const NormGeom &g, int dtype, bool bwd, NormResPlan &q)
{
    const int size = dtype == GC_F32 ? 4 : 2, widest = 16 / size;
    const bool ok = plan_small(g, widest, bwd, q) || (g.nhwc ? plan_nhwc(g, widest, size, bwd, q) : plan_nchw(g, widest, bwd, q));
    q.past = size_t(g.B) * g.img * size * (bwd ? 3 : 2) >= kStreamBytes;
    if (ok && bwd) q.ws_bytes = size_t(q.rows) * g.C * 2 * sizeof(float);
    return ok;
}
}  // namespace

// Answers are kept by shape: the search takes 0.3 to 1 us of host time, 5 us for 2048 groups
// channels last, a look into the table 0.1 to 0.2.
bool plan_norm_res(const NormGeom &g, int dtype, bool bwd, NormResPlan &q)
{
    struct Answer {
        bool ok;
        NormResPlan q;
    };
    static SearchMemo<Answer> memo;
    const int key[12] = {g.B, g.C, g.HW, g.G, g.nhwc, dtype, bwd};
    const Answer a = memo.get(key, [&] {
        Answer v{};
        v.ok = search(g, dtype, bwd, v.q);
        return v;
    });
    q = a.q;
    return a.ok;
}

}  // namespace gc

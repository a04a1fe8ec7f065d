// The index arithmetic of rows grouped by expert (grouped.hpp) on the host, its
// wave intrinsics played by 64 runs of the same code, one a lane: for right and
// for wrong offsets, where an operand's reads and writes lie.
#include <cstdint>
#include <cstdio>
#include <random>
#include <utility>
#include <vector>

namespace {
struct Dim { int x; } threadIdx;
struct Pending {};
std::vector<uint64_t> g_masks;      // of the ballots already known
std::vector<char> g_votes;          // the lanes' predicates at the next one
size_t g_call;
uint64_t ballot(bool p) {
    if (g_call < g_masks.size()) return g_masks[g_call++];
    g_votes[(size_t)threadIdx.x] = p;
    throw Pending{};
}
}  // namespace

#define __device__
#define __forceinline__ inline
#define __ballot(p) ballot(p)
#define __clzll(v) ((v) ? __builtin_clzll((unsigned long long)(v)) : 64)
#define __builtin_amdgcn_readfirstlane(v) (v)
#include "grouped.hpp"

namespace {
template <int U>
int expert_of(const int* offsets, int experts, int64_t rows, int64_t p) {
    g_masks.clear();
    for (;;) {
        g_votes.assign(64, 0);
        bool waits = false;
        int result = 0;
        for (int lane = 0; lane < 64; ++lane) {
            threadIdx.x = lane;
            g_call = 0;
            try {
                result = fp4dev::expert_of_unit<U>(offsets, experts, rows, p);
            } catch (Pending) {
                waits = true;
            }
        }
        if (!waits) return result;
        uint64_t mask = 0;
        for (int lane = 0; lane < 64; ++lane) mask |= (uint64_t)(g_votes[(size_t)lane] != 0) << lane;
        g_masks.push_back(mask);
    }
}

int g_failed = 0;
#define CHECK(c)                                                                          \
    do {                                                                                  \
        if (!(c) && ++g_failed < 20) std::printf("line %d: %s\n", __LINE__, #c);          \
    } while (0)

// What the kernels do with unit p of U rows: the expert, its rows in the unit and
// the unit's place must lie inside the tensor of `rows` rows and the operand.
template <int U>
void look(const std::vector<int>& off, int64_t rows, bool right) {
    const int experts = (int)off.size() - 1;
    const int64_t units = rows / U + experts;
    for (int64_t p = 0; p < units + 3; ++p) {
        const int e = expert_of<U>(off.data(), experts, rows, p);
        CHECK(e >= -1 && e < experts);
        if (e < 0) continue;
        const fp4dev::RowRange r = fp4dev::expert_rows(off.data(), e, rows);
        CHECK(0 <= r.lo && r.lo <= r.hi && r.hi <= rows);
        const int64_t local = p - (r.lo / U + e);
        CHECK(local >= 0);
        const int64_t first = r.lo + U * local, left = r.hi - first;
        if (left > 0) CHECK(first + (left < U ? left : U) <= rows && p < units);
        if (!right) continue;
        // the last expert that starts at or before p
        int want = -1;
        for (int i = 0; i < experts; ++i)
            if (off[(size_t)i] / U + i <= p) want = i;
        CHECK(e == want);
    }
    // an expert's span of the operand, as the products read it
    for (int e = 0; e < experts; ++e) {
        const fp4dev::RowRange r = fp4dev::expert_rows(off.data(), e, rows);
        const int64_t start = r.lo / U + e, n = (r.hi - r.lo + U - 1) / U;
        CHECK(start >= 0 && start + (n ? n : 1) <= units);
    }
}
}  // namespace

int main() {
    std::mt19937 rng(7);
    for (int turn = 0; turn < 120; ++turn) {
        const int64_t rows = 1 + rng() % (turn % 5 ? 500 : 3000);
        const int experts = turn % 40 == 7 ? 1024 : 1 + (int)(rng() % (turn % 2 ? 70 : 9));
        std::vector<int> off((size_t)experts + 1);
        const int kind = turn % 4;
        for (int& o : off) o = (int)(rng() % (uint64_t)(rows + 1));
        if (kind < 2) {
            for (size_t i = 1; i < off.size(); ++i)           // sorted: right
                for (size_t j = i; j > 0 && off[j] < off[j - 1]; --j) std::swap(off[j], off[j - 1]);
        } else if (kind == 3) {
            for (int& o : off) o = (int)rng();                // anything, also negative
        }
        look<32>(off, rows, kind < 2);
        look<256>(off, rows, kind < 2);
    }
    if (!g_failed) std::printf("ok\n");
    return g_failed != 0;
}

// A model of the K/V ring of the tensor-core chunk attention: the producer, copies
// that land in any order, the warp that looks values over, the two tiles' MMA
// threads, whose products end later than they are issued, and the slots' barriers,
// of which a wait sees the parity alone.  Every order of steps is tried.
//
//   ring_model <slots> <in_order> <rule> <part> ...
//   rule: 0 the kernels' (chunk_ring.cuh); 1 asked at a part's first fill and in
//         units of two heads; 2 at a part's first fill alone
//   part: steps,sets,steps of tile A,steps of tile B,steps whose values all rows see
//
// Prints "ok <states>", or what went wrong first.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <string>
#include <unordered_set>
#include <vector>

#include "chunk_ring.cuh"

struct Take {                // a fill that a tile's thread waits for
    int f;
    bool fixed, ask, both;   // on `fixed`; asks first; lets go of it for the other tile too
};

struct State {
    uint32_t flying = 0;             // fills begun that have not landed yet
    int8_t next = 0, spare = 0;      // fills begun (spare: no padding, a state is its bytes)
    int8_t fix = 0, fix_half = 0;    // looked over; `fixed` arrived, `empty` not yet
    int8_t took[2] = {0, 0}, freed[2] = {0, 0};
    int8_t full[8] = {}, fixed[8] = {}, empty[8] = {}, arrived[8] = {};     // phases completed; arrivals of the open one
    std::string key() const { return std::string(reinterpret_cast<const char *>(this), sizeof(*this)); }
};

static_assert(sizeof(State) == 44, "no padding");

static int slots, total;
static bool in_order;
static std::vector<Take> takes[2];
static std::string wrong;

// A wait for phase k of a barrier with c phases completed: met?
static bool met(int c, int k) { return (c & 1) != (k & 1); }

static void let_go(State &s, int f) {
    const int i = f % slots;
    if (s.empty[i] != f / slots) wrong = "a slot is let go of for fill " + std::to_string(f) + " in another phase";
    if (++s.arrived[i] == (in_order ? 2 : 3)) {
        s.arrived[i] = 0;
        ++s.empty[i];
    }
}

static void successors(const State &s, std::vector<State> &out) {
    if (s.next < total) {                                    // the producer begins a fill
        const int f = s.next, i = f % slots;
        if (met(s.empty[i], f / slots - 1)) {
            State t = s;
            ++t.next;
            t.flying |= 1u << f;
            if (t.empty[i] != f / slots) wrong = "fill " + std::to_string(f) + " begun too early";
            out.push_back(t);
        }
    }
    for (int f = 0; f < s.next; ++f)                         // one lands
        if ((s.flying >> f) & 1u) {
            State t = s;
            t.flying &= ~(1u << f);
            ++t.full[f % slots];
            out.push_back(t);
            if (in_order) break;
        }
    if (!in_order && s.fix < total) {                        // its values are looked over
        const int f = s.fix, i = f % slots;
        if (s.fix_half) {
            State t = s;
            t.fix_half = 0;
            ++t.fix;
            let_go(t, f);
            out.push_back(t);
        } else if (met(s.full[i], f / slots)) {
            State t = s;
            if (t.full[i] != f / slots + 1) wrong = "fill " + std::to_string(f) + " looked over too early";
            t.fix_half = 1;
            ++t.fixed[i];
            out.push_back(t);
        }
    }
    for (int x = 0; x < 2; ++x) {
        if (s.took[x] < (int)takes[x].size()) {              // a tile's products are issued
            const Take &u = takes[x][s.took[x]];
            const int i = u.f % slots, c = u.fixed ? s.fixed[i] : s.full[i];
            if ((!u.ask || s.next > u.f) && met(c, u.f / slots)) {
                if (c != u.f / slots + 1) {
                    wrong = "tile " + std::string(x ? "B" : "A") + " takes another fill for " + std::to_string(u.f);
                    return;
                }
                State t = s;
                ++t.took[x];
                if (u.both) let_go(t, u.f);
                out.push_back(t);
            }
        }
        if (s.freed[x] < s.took[x]) {                        // they end
            State t = s;
            let_go(t, takes[x][t.freed[x]++].f);
            out.push_back(t);
        }
    }
}

int main(int argc, char **argv) {
    if (argc < 5) return 2;
    slots = atoi(argv[1]);
    in_order = atoi(argv[2]) != 0;
    const int rule = atoi(argv[3]);
    int base = 0;
    for (int a = 4; a < argc; ++a) {
        int n, sets, steps[2], sure;
        if (sscanf(argv[a], "%d,%d,%d,%d,%d", &n, &sets, &steps[0], &steps[1], &sure) != 5) return 2;
        for (int x = 0; x < 2; ++x)
            for (int j = 0; j < steps[x]; ++j)
                for (int kv = 0; kv < 2; ++kv) {
                    const bool first = j == 0 && kv == 0;
                    const int other = sets == 2 ? 0 : steps[1 - x];
                    const bool ask = rule == 0   ? sv::chunk_ring_asks(in_order, first)
                                     : rule == 1 ? first || (sets == 2 && !in_order)
                                                 : first;
                    takes[x].push_back(Take{base + 2 * (j * sets + (sets == 2 ? x : 0)) + kv,
                                            !in_order && kv == 1 && j >= sure, ask, j >= other});
                }
        base += 2 * n * sets;
    }
    total = base;
    if (total > 31 || slots > 8) return 2;
    std::unordered_set<std::string> seen;
    std::vector<State> todo(1), next;
    seen.insert(todo[0].key());
    while (!todo.empty()) {
        const State s = todo.back();
        todo.pop_back();
        next.clear();
        successors(s, next);
        if (!wrong.empty()) {
            printf("%s\n", wrong.c_str());
            return 0;
        }
        if (next.empty() && (s.next < total || s.took[0] < (int)takes[0].size() || s.took[1] < (int)takes[1].size())) {
            printf("stuck at fill %d\n", s.next);
            return 0;
        }
        for (State &t : next)
            if (seen.insert(t.key()).second) todo.push_back(t);
        if (seen.size() > 20000000u) {
            printf("too many states\n");
            return 0;
        }
    }
    printf("ok %zu\n", seen.size());
    return 0;
}

// One warp on the host: 32 contexts that take turns, and what the split's code needs of CUDA.  Every exchange between
// lanes is a turn of all of them; the code between two exchanges runs lane by lane.  Test-side only.
#pragma once

#include <ucontext.h>

#include <algorithm>
#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <functional>
#include <vector>

#define __device__
#define __host__
#define __forceinline__ inline

namespace host_warp {

constexpr int kLanesOfWarp = 32, kStack = 64 << 10;

struct State {
    ucontext_t main, lane[kLanesOfWarp];
    std::vector<char> stacks = std::vector<char>(kLanesOfWarp * kStack);
    uint32_t value[2][kLanesOfWarp];
    int phase[kLanesOfWarp];
    bool done[kLanesOfWarp];
    int at = 0;
    std::function<void()> body;
};
inline State& state() {
    static State s;
    return s;
}
struct Index {
    unsigned x;
};
inline Index thread_index() { return Index{(unsigned)state().at}; }

inline void turn() {   // to the next lane
    State& s = state();
    const int me = s.at;
    s.at = (me + 1) % kLanesOfWarp;
    if (s.done[s.at]) abort();   // a lane left while others still exchange
    swapcontext(&s.lane[me], &s.lane[s.at]);
    s.at = me;
}
// Every lane's value, once all have given theirs.
inline const uint32_t* exchange(uint32_t v) {
    State& s = state();
    const int p = s.phase[s.at]++ & 1;
    s.value[p][s.at] = v;
    turn();
    return s.value[p];
}
inline void entry() {
    State& s = state();
    const int me = s.at;
    s.body();
    s.at = me;
    s.done[me] = true;
    if (me + 1 < kLanesOfWarp) {   // lanes end in order, after the same number of exchanges
        if (s.phase[me + 1] != s.phase[me]) abort();
        s.at = me + 1;
        setcontext(&s.lane[me + 1]);
    }
    setcontext(&s.main);
}
inline void run(const std::function<void()>& body) {
    State& s = state();
    s.body = body;
    s.at = 0;
    for (int i = 0; i < kLanesOfWarp; ++i) {
        s.phase[i] = 0;
        s.done[i] = false;
        getcontext(&s.lane[i]);
        s.lane[i].uc_stack.ss_sp = s.stacks.data() + i * kStack;
        s.lane[i].uc_stack.ss_size = kStack;
        s.lane[i].uc_link = nullptr;
        makecontext(&s.lane[i], (void (*)())entry, 0);
    }
    // the lanes start one after the other: each runs to its first exchange and hands on
    swapcontext(&s.main, &s.lane[0]);
}

}  // namespace host_warp

#define threadIdx (host_warp::thread_index())

inline int __shfl_sync(uint32_t, int v, int src) { return (int)host_warp::exchange((uint32_t)v)[src & 31]; }
inline int __shfl_up_sync(uint32_t, int v, int d) {
    const int me = (int)threadIdx.x;
    const uint32_t* all = host_warp::exchange((uint32_t)v);
    return (int)all[me >= d ? me - d : me];
}
inline int __reduce_add_sync(uint32_t, int v) {
    const uint32_t* all = host_warp::exchange((uint32_t)v);
    uint32_t sum = 0;
    for (int i = 0; i < 32; ++i) sum += all[i];
    return (int)sum;
}
inline int __reduce_max_sync(uint32_t, int v) {
    const uint32_t* all = host_warp::exchange((uint32_t)v);
    int m = (int)all[0];
    for (int i = 1; i < 32; ++i) m = std::max(m, (int)all[i]);
    return m;
}
inline unsigned __ballot_sync(uint32_t, int p) {
    const uint32_t* all = host_warp::exchange(p ? 1u : 0u);
    unsigned b = 0;
    for (int i = 0; i < 32; ++i) b |= all[i] << i;
    return b;
}
inline int __any_sync(uint32_t m, int p) { return __ballot_sync(m, p) != 0; }
inline int __ffs(unsigned x) { return __builtin_ffs((int)x); }
inline int __ldcg(const int* p) { return *p; }
inline int atomicOr(int* p, int v) {
    const int old = *p;
    *p |= v;
    return old;
}
using std::max;
using std::min;

// Model of the ring of k_act_gemm under random schedules: a producer whose loads land in any order, groups of
// warps that take the stages in turn and decode them, the MMAs.  The groups run the kernel's own walk and wait
// (csrc/ring.cuh); barriers are phases with a parity wait, as in hardware.  Every agent is a coroutine; the
// scheduler picks a random one whose wait can end, or lets a random load land.
//
//   ring_model <groups> <stages> <iterations> <quantizing 0|1> <checked 0|1> <seeds>
// prints "ok", or the first fault (a stage read before its load landed or overwritten while it was read,
// decoded twice, no agent that can go on).  checked = 0: groups that wait for full[] alone.
#include <cstdio>
#include <cstdlib>
#include <functional>
#include <memory>
#include <random>
#include <vector>

#include <ucontext.h>

#include "../qlora_parameter_efficient_b200/csrc/ring.cuh"

namespace {

const char* g_fault = nullptr;
int g_fault_it = 0;
void fault(const char* what, int it) {
    if (!g_fault) g_fault = what, g_fault_it = it;
}

struct Bar {
    int need = 1, count = 0, phase = 0;
    void arrive() {
        if (++count == need) count = 0, ++phase;
    }
    bool done(int parity) const { return (phase & 1) != parity; }
};

constexpr int kStack = 64 << 10;
ucontext_t g_main;
struct Agent {
    ucontext_t ctx;
    std::vector<char> stack = std::vector<char>(kStack);
    std::function<void()> body;
    const Bar* on = nullptr;      // waits for this barrier ...
    int parity = 0;               // ... and parity
    bool over = false;
    bool ready() const { return !over && (!on || on->done(parity)); }
};
Agent* g_now = nullptr;
void pause() { swapcontext(&g_now->ctx, &g_main); }
bool wait(const Bar& b, int parity) {
    g_now->on = &b;
    g_now->parity = parity;
    pause();
    g_now->on = nullptr;
    return !g_fault;
}
void enter() {
    g_now->body();
    g_now->over = true;
    pause();
}

struct Model {
    int G, S, n, quant, checked;
    static constexpr int kWarps = 2;                // per group
    std::vector<Bar> full, empty, decoded;
    std::vector<int> landed, tile;                  // per slot: the stage in it (-1: in flight), warps that decoded it
    struct Load { int slot, it; };
    std::vector<Load> flying;

    template <int GROUPS>
    void group_warp(int g) {
        using namespace qlora;
        RingPos at(S, g);
        auto we = [&](int i, int p) { return wait(empty[i], p); };
        auto wf = [&](int i, int p) { return wait(full[i], p); };
        for (int it = g; it < n; it += GROUPS) {
            if (checked ? !ring_landed<GROUPS>(at, we, wf) : !wf(at.s, at.ph)) return;
            if (landed[at.s] != it) return fault("read before its load landed", it);
            pause();                             // decoding takes a while
            if (landed[at.s] != it) return fault("overwritten while it was read", it);
            if (quant) {
                empty[at.s].arrive();
            } else {
                if (++tile[at.s] > kWarps) return fault("decoded too often", it);
                decoded[at.s].arrive();
            }
            at.skip(GROUPS);
        }
    }
    void producer() {
        qlora::RingPos at(S, 0);
        for (int it = 0; it < n; ++it, at.skip(1)) {
            if (!wait(empty[at.s], at.ph ^ 1)) return;
            landed[at.s] = -1;
            tile[at.s] = 0;
            flying.push_back({at.s, it});
        }
    }
    void mma() {
        qlora::RingPos at(S, 0);
        for (int it = 0; it < n; ++it, at.skip(1)) {
            if (!quant && !wait(decoded[at.s], at.ph)) return;
            if (!wait(full[at.s], at.ph)) return;
            if (landed[at.s] != it) return fault("product of a stage that has not landed", it);
            if (!quant && tile[at.s] != kWarps) return fault("product of a stage that is not decoded", it);
            pause();
            if (landed[at.s] != it) return fault("overwritten under the product", it);
            empty[at.s].arrive();
        }
    }

    bool run(unsigned seed) {
        std::mt19937 rng(seed);
        g_fault = nullptr;
        full.assign(S, Bar{});
        empty.assign(S, Bar{quant ? 1 + kWarps : 1});
        decoded.assign(S, Bar{kWarps});
        landed.assign(S, -1);
        tile.assign(S, 0);
        flying.clear();
        std::vector<std::unique_ptr<Agent>> agents;
        auto add = [&](std::function<void()> f) {
            agents.push_back(std::make_unique<Agent>());
            Agent& a = *agents.back();
            a.body = std::move(f);
            getcontext(&a.ctx);
            a.ctx.uc_stack.ss_sp = a.stack.data();
            a.ctx.uc_stack.ss_size = kStack;
            a.ctx.uc_link = nullptr;
            makecontext(&a.ctx, enter, 0);
        };
        add([this] { producer(); });
        add([this] { mma(); });
        for (int g = 0; g < G; ++g)
            for (int w = 0; w < kWarps; ++w) add([this, g] { G == 1 ? group_warp<1>(g) : G == 2 ? group_warp<2>(g) : group_warp<3>(g); });
        // how eager each agent and each load is, this time
        std::vector<int> pace(agents.size());
        for (int& p : pace) p = 1 + static_cast<int>(rng() % 20);
        const int slow = 1 + static_cast<int>(rng() % 20);
        for (;;) {
            std::vector<int> bag;
            for (size_t i = 0; i < agents.size(); ++i)
                if (agents[i]->ready()) bag.insert(bag.end(), pace[i], static_cast<int>(i));
            if (!flying.empty()) bag.insert(bag.end(), slow, -1);
            if (bag.empty()) break;
            const int k = bag[rng() % bag.size()];
            if (k < 0) {
                const size_t i = rng() % flying.size();
                landed[flying[i].slot] = flying[i].it;
                full[flying[i].slot].arrive();
                flying.erase(flying.begin() + static_cast<long>(i));
            } else {
                g_now = agents[static_cast<size_t>(k)].get();
                swapcontext(&g_main, &g_now->ctx);
            }
            if (g_fault) return false;
        }
        for (auto& a : agents)
            if (!a->over) fault("nothing can go on", -1);
        return !g_fault;
    }
};

}  // namespace

int main(int argc, char** argv) {
    if (argc != 7) return 2;
    Model m;
    m.G = atoi(argv[1]), m.S = atoi(argv[2]), m.n = atoi(argv[3]), m.quant = atoi(argv[4]), m.checked = atoi(argv[5]);
    if (m.G < 1 || m.G > 3 || m.S < m.G) return 2;
    for (int seed = 0; seed < atoi(argv[6]); ++seed)
        if (!m.run(static_cast<unsigned>(seed))) {
            printf("seed %d: %s (stage %d)\n", seed, g_fault, g_fault_it);
            return 1;
        }
    puts("ok");
    return 0;
}

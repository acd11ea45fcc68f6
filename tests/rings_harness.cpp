// The roles of the weighing kernel on modelled barriers, copies and products, in random
// schedules: the walk of its product warps (csrc/paged_rings.h) is the kernel's own,
// the other roles are written out here.  Arguments: "16" or "e4m3" (the cache), the
// walk ("kernel", or a wrong one: "skip" the other warp's key tiles, "wait" for
// them without being waited for), schedules, seed, then the units: key tiles, query
// tiles of each.  Prints how many schedules multiplied a tile that was not there, how
// many came to a standstill, and the products of one that did neither.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <deque>
#include <functional>
#include <memory>
#include <random>
#include <ucontext.h>
#include <vector>

#include "paged_rings.h"

using namespace vq;

struct Bar {  // an mbarrier: the phase completes with the last of `count` arrivals
    int count = 1, pending = 1;
    uint32_t phase = 0;
    void init(int n) { count = pending = n; }
    void arrive()
    {
        if (--pending == 0) {
            pending = count;
            ++phase;
        }
    }
    bool passed(uint32_t parity) const { return (phase & 1u) != parity; }
};

struct Sim {
    struct Role {
        ucontext_t ctx;
        std::vector<char> stack;
        std::function<void()> body;
        std::vector<std::pair<const Bar *, uint32_t>> wants;  // all of them, to go on
        bool done = false;
        double pace = 1.0;
    };
    std::mt19937 rng;
    std::vector<std::unique_ptr<Role>> roles;
    std::vector<std::function<void()>> copies;            // in flight; they land in any order
    std::vector<std::deque<std::function<void()>>> pipe;  // products and arrivals behind them, of each warp in order
    ucontext_t main_ctx;
    Role *now = nullptr;
    double copy_pace = 1.0, pipe_pace = 1.0;

    static Sim *self;
    static void enter()
    {
        Role *r = self->now;
        r->body();
        r->done = true;
        swapcontext(&r->ctx, &self->main_ctx);
    }
    void add(std::function<void()> body)
    {
        roles.emplace_back(new Role);
        Role *r = roles.back().get();
        r->body = std::move(body);
        r->stack.resize(64 * 1024);
        getcontext(&r->ctx);
        r->ctx.uc_stack.ss_sp = r->stack.data();
        r->ctx.uc_stack.ss_size = r->stack.size();
        r->ctx.uc_link = nullptr;
        makecontext(&r->ctx, enter, 0);
    }
    void yield() { swapcontext(&now->ctx, &main_ctx); }
    void wait(const Bar &a, uint32_t pa)
    {
        now->wants = {{&a, pa}};
        yield();
    }
    bool run()  // false: a standstill
    {
        self = this;
        auto pace = [&] { return rng() % 3 == 0 ? 0.02 : 1.0; };  // some are slow
        for (auto &r : roles) r->pace = pace();
        copy_pace = pace();
        pipe_pace = pace();
        for (;;) {
            std::vector<std::pair<double, int>> can;  // what may come next
            double sum = 0.0;
            auto offer = [&](double p, int what) { can.push_back({sum += p, what}); };
            bool done = copies.empty();
            for (size_t i = 0; i < roles.size(); ++i) {
                Role &r = *roles[i];
                done = done && r.done;
                bool go = !r.done;
                for (auto &w : r.wants) go = go && w.first->passed(w.second);
                if (go) offer(r.pace, (int)i);
            }
            for (size_t i = 0; i < pipe.size(); ++i)
                if (!pipe[i].empty()) offer(pipe_pace, 1000 + (int)i), done = false;
            for (size_t i = 0; i < copies.size(); ++i) offer(copy_pace / copies.size(), 2000 + (int)i);
            if (done) return true;
            if (can.empty()) return false;
            const double x = std::uniform_real_distribution<double>(0.0, sum)(rng);
            size_t c = 0;
            while (c + 1 < can.size() && can[c].first < x) ++c;
            const int what = can[c].second;
            if (what >= 2000) {
                auto f = copies[what - 2000];
                copies.erase(copies.begin() + (what - 2000));
                f();
            } else if (what >= 1000) {
                auto f = pipe[what - 1000].front();
                pipe[what - 1000].pop_front();
                f();
            } else {
                now = roles[what].get();
                now->wants.clear();
                swapcontext(&main_ctx, &now->ctx);
            }
        }
    }
};
Sim *Sim::self = nullptr;

struct Unit {
    int keys, queries;
};

enum Walk { KERNEL, SKIP, WAIT };

template <class Keys, class Queries, class Scores, class Ops>
bool wrong_products(Ops &&ops, Keys &ks, Queries &qs, Scores &ss, int g, bool two, int count, bool waits)
{
    auto pass = [&] {
        if (waits) ops.keys(ks);
        ks.step();
    };
    const bool mine = g == 0 || two;
    if (g == 1 && (two || waits)) pass();
    if (mine) ops.keys(ks);
    for (int j = 0; j < count; ++j) {
        if (mine) {
            ops.both(qs, ss);
            ops.product(ks, qs, ss);
            ss.step();
            ops.queries_used(qs);
        } else {
            ops.queries(qs);
            ops.queries_passed(qs);
        }
        qs.step();
    }
    if (mine) ops.keys_used(ks);
    if (mine || !waits) ks.step();
    if (g == 0 && two) pass();
    return true;
}

// 0: all well, 1: something was multiplied that was not there, 2: a standstill
template <bool Q8> int schedule(const std::vector<Unit> &units, Walk walk, unsigned seed, long &products)
{
    using C = WgRings<Q8>;
    constexpr int RAW = Q8 ? C::RAW : 1, CONV = Q8 ? C::CONV : 1;
    Sim sim;
    sim.rng.seed(seed);
    sim.pipe.resize(2);
    Bar k_full[C::KST], k_empty[C::KST], q_full[C::QST], q_empty[C::QST], l_full[C::LST], l_empty[C::LST], i_full[C::IST],
        i_empty[C::IST], s_full[2][C::SST], s_empty[2][C::SST], raw_full[RAW], raw_empty[RAW];
    for (auto &b : k_full) b.init(Q8 ? CONV : 1);
    for (auto &b : k_empty) b.init(walk == KERNEL ? C::READERS : 1);
    for (auto &b : q_empty) b.init(C::READERS);
    for (auto &b : l_empty) b.init(2);
    for (auto &b : i_empty) b.init(3 + 2 + (Q8 ? CONV : 0));
    for (auto &b : raw_empty) b.init(CONV);
    int keys[C::KST][CONV], queries[C::QST], raw[RAW], scores[2][C::SST][2];  // what lies there; -1: not (all of) something
    std::memset(keys, -1, sizeof(keys));
    std::memset(queries, -1, sizeof(queries));
    std::memset(raw, -1, sizeof(raw));
    bool wrong = false;
    products = 0;
    auto land = [&](int *slot, int tile, Bar &full) {
        *slot = -1;
        sim.copies.push_back([=, &full] {
            *slot = tile;
            full.arrive();
        });
    };
    auto next = [&](PgRing<C::IST> &items) {
        sim.wait(i_full[items.s], items.par);
        i_empty[items.s].arrive();
        items.step();
    };

    sim.add([&] {  // units and copies
        PgRing<C::IST> items;
        PgRing<C::KST> ks;
        PgRing<C::QST> qs;
        PgRing<RAW> rs;
        int kt = 0, qt = 0;
        for (const Unit &u : units) {
            sim.wait(i_empty[items.s], items.par ^ 1u);
            i_full[items.s].arrive();
            items.step();
            if (u.queries == 0) continue;
            for (int i = 0; i < u.keys; ++i, ++kt) {
                if (Q8) {
                    sim.wait(raw_empty[rs.s], rs.par ^ 1u);
                    land(&raw[rs.s], kt, raw_full[rs.s]);
                    rs.step();
                } else {
                    sim.wait(k_empty[ks.s], ks.par ^ 1u);
                    land(&keys[ks.s][0], kt, k_full[ks.s]);
                    ks.step();
                }
            }
            for (int j = 0; j < u.queries; ++j, ++qt) {
                sim.wait(q_empty[qs.s], qs.par ^ 1u);
                land(&queries[qs.s], qt, q_full[qs.s]);
                qs.step();
            }
        }
    });
    for (int c = 0; Q8 && c < CONV; ++c)
        sim.add([&, c] {  // codes to operands
            PgRing<C::IST> items;
            PgRing<C::KST> ks;
            PgRing<RAW> rs;
            int kt = 0;
            for (const Unit &u : units) {
                next(items);
                if (u.queries == 0) continue;
                for (int i = 0; i < u.keys; ++i, ++kt) {
                    sim.wait(raw_full[rs.s], rs.par);
                    sim.wait(k_empty[ks.s], ks.par ^ 1u);
                    if (raw[rs.s] != kt) wrong = true;
                    keys[ks.s][c] = -1;
                    sim.yield();
                    keys[ks.s][c] = kt;
                    raw_empty[rs.s].arrive();
                    k_full[ks.s].arrive();
                    rs.step();
                    ks.step();
                }
            }
        });
    for (int g = 0; g < 2; ++g)
        sim.add([&, g] {  // products
            PgRing<C::IST> items;
            PgRing<C::KST> ks;
            PgRing<C::QST> qs;
            PgRing<C::SST> ss;
            int kt = 0, qt = 0, j = 0;  // of the unit at hand: its first key and query tile, the query tile in turn
            struct Ops {
                decltype(sim) &sim_;
                std::function<bool(int)> keys_, queries_;
                std::function<bool(int, int)> both_;
                std::function<void(int, int, int)> product_;
                Bar *k_empty_, *q_empty_;
                int g_;
                bool keys(const PgRing<C::KST> &k) { return keys_(k.s + 16 * (int)k.par); }
                bool queries(const PgRing<C::QST> &q) { return queries_(q.s + 16 * (int)q.par); }
                bool both(const PgRing<C::QST> &q, const PgRing<C::SST> &s) { return both_(q.s + 16 * (int)q.par, s.s + 16 * (int)s.par); }
                void product(const PgRing<C::KST> &k, const PgRing<C::QST> &q, const PgRing<C::SST> &s) { product_(k.s, q.s, s.s); }
                void used(Bar *b) { sim_.pipe[g_].push_back([b] { b->arrive(); }); }
                void keys_used(const PgRing<C::KST> &k) { used(k_empty_ + k.s); }
                void queries_used(const PgRing<C::QST> &q) { used(q_empty_ + q.s); }
                void keys_passed(const PgRing<C::KST> &k) { k_empty_[k.s].arrive(); }
                void queries_passed(const PgRing<C::QST> &q) { q_empty_[q.s].arrive(); }
            };
            Ops ops{sim,
                    [&](int k) { sim.wait(k_full[k & 15], (uint32_t)(k >> 4)); return true; },
                    [&](int q) { sim.wait(q_full[q & 15], (uint32_t)(q >> 4)); return true; },
                    [&](int q, int s) {
                        sim.wait(q_full[q & 15], (uint32_t)(q >> 4));
                        sim.wait(s_empty[g][s & 15], (uint32_t)(s >> 4) ^ 1u);
                        return true;
                    },
                    [&](int k, int q, int s) {
                        const int key = kt + g, query = qt + j++;
                        sim.pipe[g].push_back([&, k, q, s, key, query] {
                            for (int c = 0; c < CONV; ++c) wrong = wrong || keys[k][c] != key;
                            wrong = wrong || queries[q] != query;
                            scores[g][s][0] = key;
                            scores[g][s][1] = query;
                            ++products;
                            s_full[g][s].arrive();
                        });
                    },
                    k_empty, q_empty, g};
            for (const Unit &u : units) {
                next(items);
                if (u.queries == 0) continue;
                j = 0;
                if (walk == KERNEL) wg_products(ops, ks, qs, ss, g, u.keys == 2, u.queries);
                else wrong_products(ops, ks, qs, ss, g, u.keys == 2, u.queries, walk == WAIT);
                kt += u.keys;
                qt += u.queries;
            }
        });
    sim.add([&] {  // the rows' -lse
        PgRing<C::IST> items;
        PgRing<C::LST> ls;
        for (const Unit &u : units) {
            next(items);
            for (int j = 0; j < u.queries; ++j) {
                sim.wait(l_empty[ls.s], ls.par ^ 1u);
                l_full[ls.s].arrive();
                ls.step();
            }
        }
    });
    for (int g = 0; g < 2; ++g)
        sim.add([&, g] {  // sums
            PgRing<C::IST> items;
            PgRing<C::LST> ls;
            PgRing<C::SST> ss;
            int kt = 0, qt = 0;
            for (const Unit &u : units) {
                next(items);
                for (int j = 0; j < u.queries; ++j) {
                    sim.wait(l_full[ls.s], ls.par);
                    if (g < u.keys) {
                        sim.wait(s_full[g][ss.s], ss.par);
                        wrong = wrong || scores[g][ss.s][0] != kt + g || scores[g][ss.s][1] != qt + j;
                        s_empty[g][ss.s].arrive();
                        ss.step();
                    }
                    l_empty[ls.s].arrive();
                    ls.step();
                }
                if (u.queries > 0) {
                    kt += u.keys;
                    qt += u.queries;
                }
            }
        });
    const bool finished = sim.run();
    return wrong ? 1 : finished ? 0 : 2;
}

int main(int argc, char **argv)
{
    if (argc < 7) return 2;
    const bool q8 = std::strcmp(argv[1], "e4m3") == 0;
    const Walk walk = std::strcmp(argv[2], "skip") == 0 ? SKIP : std::strcmp(argv[2], "wait") == 0 ? WAIT : KERNEL;
    const int runs = std::atoi(argv[3]);
    const unsigned seed = (unsigned)std::atoi(argv[4]);
    std::vector<Unit> units;
    for (int i = 5; i + 1 < argc; i += 2) units.push_back({std::atoi(argv[i]), std::atoi(argv[i + 1])});
    int bad[3] = {0, 0, 0};
    long products = 0, n = 0;
    for (int r = 0; r < runs; ++r) {
        const int x = q8 ? schedule<true>(units, walk, seed + r, n) : schedule<false>(units, walk, seed + r, n);
        ++bad[x];
        if (x == 0) products = n;
    }
    std::printf("%d %d %ld\n", bad[1], bad[2], products);
    return 0;
}

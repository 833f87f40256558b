/*
 * The ring of copies of the norm's gradient, stopped at every point: a model of its places' mbarriers and of its loop (a
 * thread that issues, threads that wait, a wait that runs out, the loop going on without copies), and the waits that the
 * kernel makes before it leaves (csrc/bulk_ring.cuh).  Prints what went wrong, and returns 1, if a copy is still under
 * way after them or one of them names a phase that no copy completes.
 */
#include <cstdio>
#include <cstring>
#include <vector>

#include "bulk_ring.cuh"

struct Place {
    unsigned phase = 0;          // the phase that is not complete
    bool armed = false;          // a copy is on its way to it
    void issue() { armed = true; }
    void land()
    {
        if (armed) ++phase, armed = false;
    }
    // what a wait with this parity finds: complete, completed by the copy under way, or neither
    enum Found { kThere, kComes, kNever };
    Found wait(unsigned parity) const
    {
        return (phase & 1u) != parity ? kThere : armed ? kComes : kNever;
    }
};

/* by_count: the waits as the loop's own count of places has them, for comparison */
static int stopped(unsigned slots, unsigned mine, unsigned stop, bool issuer_waited, bool by_count)
{
    std::vector<Place> places(slots);
    unsigned issued = 0, slot = 0, phase = 0;
    bool abort = false;
    for (unsigned i = 0; i < slots && i < mine; ++i, ++issued) places[i].issue();
    for (unsigned g = 0; g < mine; ++g) {
        /* from group `stop` on a copy lands only when it is waited for at the end; at `stop` itself the issuing thread
           may have seen it while another gave up */
        if (g < stop || (g == stop && issuer_waited && !abort)) {
            if (places[slot].wait(phase) == Place::kNever) return 2;      /* the model's own loop */
            if (places[slot].wait(phase) == Place::kComes) places[slot].land();
        }
        if (g >= stop) abort = true;
        if (g > 0 && g - 1 + slots < mine && !abort) {
            places[(g - 1) % slots].issue();
            ++issued;
        }
        if (++slot == slots) slot = 0, phase ^= 1u;
    }
    unsigned wrong = 0;
    if (by_count) {
        for (unsigned i = 0; i < slots; ++i) {
            const Place::Found f = places[i].wait(phase ^ (i < slot ? 1u : 0u));
            wrong += f == Place::kNever;
            if (f == Place::kComes) places[i].land();
        }
    } else {
        for (unsigned x = moe::ring_first_open(issued, slots); x < issued; ++x) {
            Place &p = places[moe::ring_place(x, slots)];
            const Place::Found f = p.wait(moe::ring_parity(x, slots));
            wrong += f == Place::kNever;
            if (f == Place::kComes) p.land();
        }
    }
    for (const Place &p : places) wrong += p.armed;
    return wrong ? 1 : 0;
}

int main(int argc, char **argv)
{
    const bool by_count = argc > 1 && !strcmp(argv[1], "by_count");
    unsigned cases = 0, bad = 0;
    for (unsigned slots = 2; slots <= 8; ++slots)
        for (unsigned mine = 1; mine <= 5 * slots + 3; ++mine)
            for (unsigned stop = 0; stop <= mine; ++stop)
                for (int issuer = 0; issuer < 2; ++issuer) {
                    const int r = stopped(slots, mine, stop, issuer != 0, by_count);
                    ++cases;
                    if (!r) continue;
                    if (bad++ < 5) printf("slots %u, groups %u, stopped at %u, issuer waited %d: %s\n", slots, mine, stop, issuer, r == 2 ? "model" : "wrong");
                }
    printf("%u cases, %u wrong\n", cases, bad);
    return bad != 0;
}

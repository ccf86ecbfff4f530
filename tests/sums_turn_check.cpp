// Checks SumsTurn (csrc/ep_sums_turn.cuh) on sequences of tiles: what its waits prove to be done, and nothing else, is
// taken as done. Two groups of warps read the sums as the kernel's do, as late as the waits allow. Prints the first
// sequence in which a block's sums would overwrite columns that a group may still read, or in which a wait never ends.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "ep_sums_turn.cuh"

namespace {

struct Tile {
    bool lanes;
    int blocks;
};

// Places in a group's program: how many of its reads have been issued for, how many are proven to be done.
struct Group {
    int reads = 0, done = 0;
};

struct Model {
    Group groups[2];
    int last[ep::kBuffers][2][2] = {};              // buffer, half of 64 columns, group: its last read of them (1 and up)
    std::vector<int> announced[ep::kBuffers];       // by phase: the announcing group's read ...
    std::vector<int> announcer[ep::kBuffers];       // ... and the group
    int known[ep::kBuffers] = {};                   // phases proven to be complete
    const char* fault = nullptr;

    void wait(int buffer, uint32_t parity) {
        // The fewest phases with which a wait for this parity ends: it does where the last complete one has it.
        int n = known[buffer];
        if (((static_cast<uint32_t>(n) + 1) & 1) != parity) ++n;
        if (n > static_cast<int>(announced[buffer].size())) {
            fault = "a wait that never ends";
            return;
        }
        known[buffer] = n;
        for (int k = 0; k < n; ++k) {
            Group& g = groups[announcer[buffer][k]];
            if (announced[buffer][k] > g.done) g.done = announced[buffer][k];
        }
    }
    void write(int buffer, int half) {
        for (int g = 0; g < 2; ++g)
            if (last[buffer][half][g] > groups[g].done) fault = "sums over columns that may still be read";
    }
    void read(int group, int buffer, int half) { last[buffer][half][group] = groups[group].reads; }
    void announce(int group, int buffer) {
        announced[buffer].push_back(groups[group].reads);
        announcer[buffer].push_back(group);
    }
};

const char* run(const std::vector<Tile>& tiles) {
    ep::SumsTurn turn;
    Model m;
    for (const Tile& t : tiles) {
        for (int b = 0; b < t.blocks; ++b) {
            const int at = turn.next(t.lanes, [&](int buffer, uint32_t parity) { m.wait(buffer, parity); });
            if (t.lanes && at % 2 != 0) return "a pair that starts at an odd buffer";
            for (int half = 0; half < 2; ++half)
                for (int k = 0; k < (t.lanes ? 2 : 1); ++k) m.write(at + k, half);
            if (m.fault) return m.fault;
            if (t.lanes) {
                for (int g = 0; g < 2; ++g) {
                    ++m.groups[g].reads;
                    m.read(g, at, g);
                    m.read(g, at + 1, g);
                    m.announce(g, at + g);
                }
            } else {
                const int g = b % 2;
                ++m.groups[g].reads;
                m.read(g, at, 0);
                m.read(g, at, 1);
                m.announce(g, at);
            }
        }
    }
    return nullptr;
}

bool ok(const std::vector<Tile>& tiles) {
    const char* fault = run(tiles);
    if (!fault) return true;
    std::printf("%s:", fault);
    for (const Tile& t : tiles) std::printf(" %s %d", t.lanes ? "lanes" : "columns", t.blocks);
    std::printf("\n");
    return false;
}

// All sequences of up to `more` further tiles of 1 to 5 blocks.
bool all(std::vector<Tile>& tiles, int more) {
    if (!ok(tiles)) return false;
    if (more == 0) return true;
    for (int k = 0; k < 10; ++k) {
        tiles.push_back({k % 2 == 1, 1 + k / 2});
        const bool fine = all(tiles, more - 1);
        tiles.pop_back();
        if (!fine) return false;
    }
    return true;
}

}  // namespace

int main() {
    std::vector<Tile> tiles;
    if (!all(tiles, 5)) return 1;
    std::srand(1);
    for (int n = 0; n < 2000; ++n) {
        tiles.clear();
        for (int k = 0; k < 60; ++k) tiles.push_back({std::rand() % 2 == 1, 1 + std::rand() % 12});
        if (!ok(tiles)) return 1;
    }
    std::printf("ok\n");
    return 0;
}

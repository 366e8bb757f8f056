// q4k_maps.h -- where a host thread keeps its encoded tensor maps: the key of a map
// and its place. Plain C++.
#pragma once

#include <stdint.h>

namespace q4k {

// A map is a pure function of the base address, the tensor's dimensions and the box
// (everything else is fixed per kind): 0 packed weights, 1 rows of the dense GEMM, 2 of the experts'.
struct MapKey {
    uintptr_t ptr;
    int64_t a, b;
    int box, kind;
    bool operator==(const MapKey& o) const {
        return ptr == o.ptr && a == o.a && b == o.b && box == o.box && kind == o.kind;
    }
};
constexpr int kMapCacheSize = 1024;

// The place of a map in a cache of kMapCacheSize. Boxes (of up to 256 rows, in steps of
// 16) and kinds of the same array lie side by side: a call that takes several of them finds all
// of them again.
inline unsigned map_slot_index(const MapKey& k) {
    uint64_t h = static_cast<uint64_t>(k.ptr >> 4) * 0x9E3779B97F4A7C15ull;
    h ^= static_cast<uint64_t>(k.a) * 0xBF58476D1CE4E5B9ull;
    h ^= static_cast<uint64_t>(k.b) * 0x94D049BB133111EBull;
    return static_cast<unsigned>(((h >> 40) + 17 * k.kind + k.box / 16) % kMapCacheSize);
}

}  // namespace q4k

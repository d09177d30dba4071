// mx_fp4_choice.h -- tile, split and grid of a 4-bit product, by its sizes and the device's SMs.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>

namespace mx {
namespace fp4 {

// Token tile, cluster split and grid of a product.
struct Choice {
    int nt, cl, grid;
    bool several;  // tiles to a CTA
};

// Rounds of `units` tiles over the SMs, each as long as the MMAs of `rows` tokens and about 40 tokens' worth besides.
inline double rounds(double units, double rows, int sms) { return std::ceil(units / sms) * (rows + 40); }

inline Choice choose(int rows, bool grouped, int E, int FT, int KB, int sms)
{
    Choice c{16, 1, 1, true};
    if (grouped) {
        // The smallest tile that holds a group with as many rows as an even routing gives; of many rows that whose
        // rounds take least (a group of other sizes ends with half a tile on average).  An empty part of a tile
        // costs shared memory alone: 4096 rows of 128 matrices 704 x 2816 by 64, 128 and 224 29.1, 28.8 and 31.7 us;
        // 32768 of 256 matrices 1024 x 4096 140, 121 and 119; 4096 of 8 such 18.5, 15.0 and 18.4.
        const double avg = (double)rows / E, most = avg + 3 * std::sqrt(avg);
        for (int nt : {32, 64})
            if (c.nt < most)
                c.nt = nt;
        double best = 1e30;
        if (most > 64)
            for (int nt : {64, 128, 224}) {
                const double tiles = most <= nt ? 1.0 : avg / nt + 0.5;
                const double t = rounds(E * tiles * FT, avg / tiles, sms);
                if (t < best)
                    best = t, c.nt = nt;
            }
        const int64_t units = ((int64_t)rows / c.nt + E) * FT;
        c.grid = (int)std::min<int64_t>(sms, units);
        return c;
    }
    for (int nt : {32, 64})
        if (c.nt < rows)
            c.nt = nt;
    auto units_of = [&](int nt) { return (int64_t)((rows + nt - 1) / nt) * FT; };
    if (rows > 64 && 2 * units_of(64) > sms) {
        double best = 1e30;
        for (int nt : {64, 128, 224}) {
            const double t = rounds((double)units_of(nt), nt, sms);
            if (t < best)
                best = t, c.nt = nt;
        }
    }
    // Few units of many stages: clusters of four split the inner dimension, of eight where a few such clusters do.  A
    // cluster costs 1 to 1.5 us: 20 x 4096 x 4096 (16 stages, blocks of 16) whole 6.2 us, in four 6.0, 64 rows 6.6, 6.8; 2112 x 5120 6.8, 5.9 and
    // 7.3, 6.8; 4096 x 2048 4.8, 5.3.  In two it gains nothing while more do not fit (20 x 7680 x 8192 9.9 and 10.0 us), and 17
    // units in eight wait for room (a GPC holds one or two clusters of eight; 20 x 2112 x 8192 10.9 us, in four 6.4).  A
    // cluster has one unit: the kernel keeps no partial sums of a second.
    const int64_t units = units_of(c.nt);
    if (units <= 8 && 8 * units <= sms && KB >= 16)
        c.cl = 8;
    else if (4 * units <= sms && KB >= (rows <= 32 ? 16 : 18))
        c.cl = 4;
    c.grid = (int)std::min<int64_t>(sms / c.cl, units) * c.cl;
    c.several = units > c.grid / c.cl;
    return c;
}

}  // namespace fp4
}  // namespace mx

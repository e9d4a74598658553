// rope_table.cpp -- the rotary table (w12_rope_table), on the host in double
// precision: a model makes it once, and the angle p * f keeps its low bits at
// any position (an fp32 product is off by 2^-24 of a large angle).
#include <cmath>

#include "../../include/w12.h"

namespace {

constexpr double kPi = 3.14159265358979323846;
constexpr int kPairs = 512;  // channel pairs at a time: their frequencies are on the stack

double clamp01(double x) { return x < 0.0 ? 0.0 : x > 1.0 ? 1.0 : x; }

}  // namespace

extern "C" int w12_rope_table(int64_t positions, int rot, double base, const w12_rope_scaling *sc, float *table) {
    if (positions < 0 || rot < 8 || rot % 8 != 0) return W12_ERR_SHAPE;
    const int mode = sc ? sc->mode : W12_ROPE_SCALE_NONE;
    if (!(base > 1.0) || !std::isfinite(base) || mode < W12_ROPE_SCALE_NONE || mode > W12_ROPE_SCALE_YARN)
        return W12_ERR_ARG;
    if (mode != W12_ROPE_SCALE_NONE && !(sc->factor > 0.0 && std::isfinite(sc->factor))) return W12_ERR_ARG;
    const bool bands = mode == W12_ROPE_SCALE_BANDS || mode == W12_ROPE_SCALE_YARN;
    if (bands && !(sc->original > 0.0 && std::isfinite(sc->original) && sc->low > 0.0 && sc->high > sc->low &&
                   std::isfinite(sc->high)))
        return W12_ERR_ARG;
    if (mode == W12_ROPE_SCALE_YARN && !(sc->attention >= 0.0 && std::isfinite(sc->attention))) return W12_ERR_ARG;
    if (positions == 0) return W12_OK;
    if (!table) return W12_ERR_ARG;

    const int half = rot / 2;
    double f[kPairs], amp = 1.0, b = base, j0 = 0.0, j1 = 0.0;
    if (mode == W12_ROPE_SCALE_BASE) b = base * std::pow(sc->factor, double(rot) / double(rot - 2));
    if (mode == W12_ROPE_SCALE_YARN) {
        // channel pair that makes t turns over the original length
        const auto pair_at = [&](double t) {
            return rot * std::log(sc->original / (2.0 * kPi * t)) / (2.0 * std::log(base));
        };
        j0 = std::fmax(std::floor(pair_at(sc->high)), 0.0);
        j1 = std::fmin(std::ceil(pair_at(sc->low)), double(rot - 1));
        if (j1 <= j0) j1 = j0 + 0.001;
        amp = sc->attention > 0.0 ? sc->attention : 0.1 * std::log(sc->factor) + 1.0;
    }
    for (int first = 0; first < half; first += kPairs) {
        const int n = half - first < kPairs ? half - first : kPairs;
        for (int i = 0; i < n; ++i) {
            const int j = first + i;
            double v = std::pow(b, -2.0 * j / rot);
            if (mode == W12_ROPE_SCALE_LINEAR) v /= sc->factor;
            if (bands) {
                const double g = mode == W12_ROPE_SCALE_BANDS
                                     ? clamp01((sc->original * v / (2.0 * kPi) - sc->low) / (sc->high - sc->low))
                                     : 1.0 - clamp01((j - j0) / (j1 - j0));
                v = v * g + v / sc->factor * (1.0 - g);
            }
            f[i] = v;
        }
#pragma omp parallel for schedule(static)
        for (int64_t p = 0; p < positions; ++p) {
            float *t = table + p * rot + first;
            for (int i = 0; i < n; ++i) {
                t[i] = float(std::cos(double(p) * f[i]) * amp);
                t[half + i] = float(std::sin(double(p) * f[i]) * amp);
            }
        }
    }
    return W12_OK;
}

"""Plain stores of staged logits, lane by lane on the CPU: what they read lies in
the boxes that one warp stages, what they write is every logit of its rows once."""
import re

import pytest

import device_text as D

SHIM = r"""
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <vector>
#define __device__
#define __forceinline__ inline
struct uint4 { uint32_t x, y, z, w; };
static uint4 make_uint4(uint32_t x, uint32_t y, uint32_t z, uint32_t w) { return {x, y, z, w}; }
static uint32_t __byte_perm(uint32_t a, uint32_t b, uint32_t s)
{
    const uint64_t v = (uint64_t(b) << 32) | a;
    uint32_t r = 0;
    for (int i = 0; i < 4; ++i)
        r |= uint32_t((v >> (8 * ((s >> (4 * i)) & 7))) & 0xFF) << (8 * i);
    return r;
}
constexpr int kL8BoxBytes = 2048;
struct Lm8Params { int32_t M, N; uint16_t *logits; };
static std::vector<uint8_t> staged(1 << 16);
static uint32_t least = ~0u, most = 0;
static uint4 l8_staged4(uint32_t a)
{
    least = a < least ? a : least;
    most = a + 16 > most ? a + 16 : most;
    uint4 r;
    memcpy(&r, &staged[a], 16);
    return r;
}
static uint16_t l8_staged1(uint32_t a)
{
    least = a < least ? a : least;
    most = a + 2 > most ? a + 2 : most;
    uint16_t r;
    memcpy(&r, &staged[a], 2);
    return r;
}
"""

MAIN = r"""
int main()
{
    constexpr uint32_t base = 16384;
    for (int N : {33, 96, 97, 99, 200, 203})
        for (int ncols : {1, 5, 7, 8, 9, 31, 32, 63, 64, 65, 90, 95, 96, 127, 128})
            for (int off = 0; off < 8; ++off)
                for (int M : {1, 2, 5, 31, 32, 40}) {
                    if (ncols > 32 * BOXES || ncols > N)
                        continue;
                    const int rows = M < 32 ? M : 32, n = N - ncols;
                    std::vector<uint16_t> out(static_cast<size_t>(M) * N + 64, 0xFFFF);
                    uint16_t *p = out.data();
                    while ((reinterpret_cast<uintptr_t>(p) & 15) != 0)
                        ++p;
                    p += off;
                    std::fill(staged.begin(), staged.end(), 0xEE);
                    for (int r = 0; r < 32; ++r)
                        for (int c = 0; c < 32 * BOXES; ++c) {
                            const uint16_t v = static_cast<uint16_t>(r * 128 + c);
                            memcpy(&staged[l8_staged_at(base, r, c)], &v, 2);
                        }
                    Lm8Params P = {M, N, p};
                    for (int lane = 0; lane < 32; ++lane)
                        CALL(P, base, 0, n, ncols, lane);
                    for (uint16_t *q = out.data(); q < out.data() + out.size(); ++q) {
                        const long long i = q - p, r = i >= 0 ? i / N : -1, c = i >= 0 ? i % N - n : -1;
                        const bool in = r >= 0 && r < rows && c >= 0 && c < ncols;
                        if (*q != (in ? static_cast<uint16_t>(r * 128 + c) : 0xFFFF)) {
                            printf("wrong: N %d ncols %d off %d M %d at %lld %lld\n", N, ncols, off, M, r, c);
                            return 0;
                        }
                    }
                }
    printf("%s %u %u\n", least >= base && most <= base + BOXES * kL8BoxBytes ? "inside" : "outside", least - base, most - base);
}
"""


@pytest.mark.parametrize("file,boxes", [("sv_lmhead_fp4.cuh", 3), ("sv_lmhead_fp8.cuh", 4)])
def test_reads_stay_in_a_warps_boxes(file, boxes, tmp_path):
    text = open(f"{D.CSRC}/{file}", encoding="utf-8").read()
    call = re.findall(r"\b(l8_store_rows(?:<[^>]*>)?)\((?:P|T), ", text)
    assert call
    code = SHIM + "#include <algorithm>\nconstexpr int kL4MaxNB = 192;\n" + f"constexpr int BOXES = {boxes};\n"
    code += "".join(D.function("sv_lmhead_fp8.cuh", f) for f in ("l8_staged_at", "l8_shift", "l8_store_rows"))
    out = D.run(code + f"#define CALL {call[0]}\n" + MAIN, tmp_path)
    assert out.startswith("inside"), out

// Host check of the cache's stored values: every bf16 pattern under a range of scale exponents, and every e4m3 byte
// moved down by every shift, through the functions that the kernels use.  Writes two tables that
// test_cache_math.py compares with the definitions.
#include <cstdio>

#include "cache.cuh"

int main(int argc, char** argv) {
    if (argc != 2) return 2;
    FILE* f = fopen(argv[1], "wb");
    if (!f) return 2;
    const int exps[] = {-100, -20, -14, -9, -8, -7, -1, 0, 5, 60, 119, 120};
    for (int E : exps)
        for (unsigned h = 0; h < 65536; ++h) {
            const unsigned char b = (unsigned char)tbik::cache_quant(h, E);
            fwrite(&b, 1, 1, f);
        }
    for (unsigned h = 0; h < 0x7F80; ++h) {
        const int E = tbik::cache_need(tbik::cache_round4(h));
        fwrite(&E, 4, 1, f);
    }
    for (int d = 0; d <= 40; ++d)
        for (unsigned q = 0; q < 256; ++q) {
            const unsigned char b = (unsigned char)tbik::cache_down(q, d);
            fwrite(&b, 1, 1, f);
        }
    return fclose(f) ? 1 : 0;
}

// product_shape.h -- which shape of tiles an experts' product or gradient takes, by
// its sizes; plain C++, not exported.
#pragma once

#include <cstddef>

namespace hr {

enum class ProductShape { Large, Half, Middle, Some, Low, Few, FewAcross, Tiny, AnyMiddle, AnyFew };
enum class GradientShape { Large, Middle, Deep, AnyMiddle };

// Tiles that segments of so many rows in all take at most.
inline size_t tiles_of(size_t rows, int experts, size_t high) {
    const size_t used = static_cast<size_t>(experts) < rows ? experts : rows;
    const size_t most = rows / high + used;
    return most < rows ? most : rows;
}

// The largest shape whose height fits the segments and whose tiles fill the GPU.
// (The rows are the buffer's: with padded segments more than there are.)  us by
// shape, the chosen one first.
// 4096 x 4096, bfloat16, one matrix: 16 rows Tiny 7.2 Few 8.0; 64 Few 12.2 Low
// 21.4; 256 Low 22.9 Some 32.1 Few 39; 512 Some 33.8 Low 43 Middle 43; 1024 Some
// 42.8 Middle 47 Half 60; 2048 Middle 63.9 Half 66.0 large 78; 4096 large 98
// Middle 133 Half 138.
// 64 matrices of 2048 x 4096, rows per matrix on average 8: Few 157 Some 162; 16: Low
// 179 Middle 170 Few 196; 32: Some 192 Middle 175 Few 272; 47 with padding: Middle
// 176 Half 183 Some 192; 64: Half 224 large 210 Middle 236; 128: Half 268 large 293;
// 256: large 372 Half 391.  e4m3: 8: Few 86 Some 105; 16: Low 115 Some 114 Middle
// 125; 32: Some 121 Middle 125; 47: Middle 126 Some 119; 64: Half 144 Some 136; 128:
// Half 173 large 206; 256: large 255 Half 266.
// 64 matrices of 2560 x 5120 and padding to 16 rows, 512 rows in 1472: Some 264 Low 254
// Middle 299 Few 279; 1024 in 1984: Some 283 Low 285 Middle 310.
// Transposed 2 rows: FewAcross 10.3 Low 21; e4m3 512 rows of 64: Low 93 FewAcross 123.
inline ProductShape product_shape(size_t rows, int experts, size_t n, bool across, bool any) {
    const size_t each = rows / experts;
    const auto fits = [&](size_t bq, size_t bp, size_t least_rows, size_t least_tiles) {
        return each >= least_rows && tiles_of(rows, experts, bq) * ((n + bp - 1) / bp) >= least_tiles;
    };
    if (any) return fits(128, 128, 24, 128) ? ProductShape::AnyMiddle : ProductShape::AnyFew;
    if (fits(256, 256, 192, 200)) return ProductShape::Large;
    if (fits(128, 256, 64, 320)) return ProductShape::Half;
    if (fits(128, 128, 40, 320)) return ProductShape::Middle;
    if (fits(64, 128, 20, 200)) return ProductShape::Some;
    if (fits(32, 128, 12, 128)) return ProductShape::Low;
    if (across) return fits(32, 128, 0, 256) ? ProductShape::Low : ProductShape::FewAcross;
    return fits(16, 32, 0, 192) ? ProductShape::Few : ProductShape::Tiny;
}

// Segments differ in length: one round of large tiles is as long as the longest.  32
// matrices of 1024 x 512 over 32768 rows, 256 large tiles 77 us, 1024 of Middle 56;
// 1024 x 1024 93 and 101; one matrix has no such difference.
inline GradientShape gradient_shape(int experts, size_t n, size_t k, bool any) {
    if (any) return GradientShape::AnyMiddle;
    const auto tiles = [&](size_t b) { return ((n + b - 1) / b) * ((k + b - 1) / b) * experts; };
    if (n >= 192 && k >= 192 && tiles(256) >= (experts > 1 ? 400u : 200u)) return GradientShape::Large;
    return tiles(128) >= 320 ? GradientShape::Middle : GradientShape::Deep;
}

}  // namespace hr

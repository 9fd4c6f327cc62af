/*
 * A plain C11 client of the entry points of include/fp8bs.h between a step's
 * linears and its attention (norm and rotation into the caches, routing and
 * combination of experts, sampling): takes the address of each (a missing
 * export fails the link) and checks their argument validation through the C
 * calling convention.  Every call here is refused, or has nothing to do,
 * before the library touches CUDA, so no GPU is needed.  Prints
 * "checks <n> failures <f>" and exits non-zero on any failure.
 */
#include <stdint.h>
#include <stdio.h>

#include "fp8bs.h"

static int checks, failures;

static void expect(int64_t got, int64_t want, const char *what, int line)
{
    ++checks;
    if (got != want) {
        ++failures;
        printf("FAIL line %d: %s returned %lld, expected %lld\n", line, what, (long long)got, (long long)want);
    }
}
#define EXPECT(call, want) expect((call), (want), #call, __LINE__)

/* fake, never dereferenced device addresses */
#define P(type, v) ((type *)(uintptr_t)(v))

/* one call's arguments; a test changes one of them */
struct rope {
    int64_t tokens, hq, hkv, dim, stride, max_pos, rot, page, blocks;
    const void *q;
    const int32_t *pos;
    float eps;
    uint8_t *cache;
};

static int run_rope8(struct rope r)
{
    return fp8kv_rope_append(r.q, r.stride, r.q, r.stride, r.q, r.stride, r.tokens, r.hq, r.hkv, r.dim, r.pos, r.pos,
                             P(float, 0x10000), r.max_pos, r.rot, 0, NULL, NULL, r.eps, P(void, 0x20000),
                             P(float, 0x30000), P(float, 0x30000), r.cache, r.cache, r.page * r.blocks, NULL);
}

static int run_rope4(struct rope r)
{
    return fp4kv_rope_append(r.q, r.stride, r.q, r.stride, r.q, r.stride, r.tokens, r.hq, r.hkv, r.dim, r.pos, r.pos,
                             P(float, 0x10000), r.max_pos, r.rot, 1, NULL, NULL, r.eps, P(void, 0x20000),
                             P(float, 0x30000), P(float, 0x30000), r.cache, r.cache, r.page, r.blocks, NULL);
}

struct route {
    int64_t stride, tokens, experts, topk, groups, open, top;
    int f32, scoring;
    const void *x;
    int32_t *ids;
    float scale;
};

static int run_route(struct route r)
{
    return fp8bs_moe_route(r.x, r.f32, r.stride, r.tokens, r.experts, r.topk, r.scoring, NULL, r.groups, r.open, r.top, 1,
                           r.scale, r.ids, P(float, 0x50000), NULL);
}

struct comb { int64_t experts, tokens, topk, n; const void *y; const int32_t *ids; void *out; };

static int run_comb(struct comb c)
{
    return fp8bs_moe_combine(c.y, P(float, 0x10000), c.ids, c.experts, NULL, c.tokens, c.topk, c.n, c.out, NULL);
}

struct draw { int64_t stride, rows, vocab; int f32; const void *x; const float *u; int32_t *tokens; };

static int run_draw(struct draw d)
{
    return fp8bs_sample_tokens(d.x, d.f32, d.stride, d.rows, d.vocab, d.u, NULL, NULL, NULL, NULL, d.tokens, NULL, NULL);
}

#define WITH(type, base, field, value) ((void)0, (tmp_##type = base, tmp_##type.field = value, tmp_##type))

int main(void)
{
    struct rope tmp_rope;
    struct route tmp_route;
    struct comb tmp_comb;
    struct draw tmp_draw;

    /* norm, rotation and cache write */
    const struct rope r = {4, 8, 2, 128, 1024, 64, 128, 16, 64, P(void, 0x40000), P(int32_t, 0x50000), 1e-6f,
                           P(uint8_t, 0x60000)};
    int (*const ropes[2])(struct rope) = {run_rope8, run_rope4};
    for (int i = 0; i < 2; ++i) {
        EXPECT(ropes[i](WITH(rope, r, tokens, -1)), FP8BS_ERR_SHAPE);
        EXPECT(ropes[i](WITH(rope, r, hq, 0)), FP8BS_ERR_SHAPE);
        EXPECT(ropes[i](WITH(rope, r, hkv, 0)), FP8BS_ERR_SHAPE);
        EXPECT(ropes[i](WITH(rope, r, dim, 96)), FP8BS_ERR_SHAPE);
        EXPECT(ropes[i](WITH(rope, r, rot, 24)), FP8BS_ERR_SHAPE);
        EXPECT(ropes[i](WITH(rope, r, rot, 144)), FP8BS_ERR_SHAPE);
        EXPECT(ropes[i](WITH(rope, r, max_pos, 0)), FP8BS_ERR_SHAPE);
        EXPECT(ropes[i](WITH(rope, r, blocks, 0)), FP8BS_ERR_SHAPE);
        EXPECT(ropes[i](WITH(rope, r, eps, -1.0f)), FP8BS_ERR_SHAPE);
        EXPECT(ropes[i](WITH(rope, r, stride, 1028)), FP8BS_ERR_ALIGN);
        EXPECT(ropes[i](WITH(rope, r, q, NULL)), FP8BS_ERR_NULL);
        EXPECT(ropes[i](WITH(rope, r, q, P(void, 0x40008))), FP8BS_ERR_ALIGN);
        EXPECT(ropes[i](WITH(rope, r, pos, P(int32_t, 0x50002))), FP8BS_ERR_ALIGN);
        EXPECT(ropes[i](WITH(rope, r, cache, NULL)), FP8BS_ERR_NULL);
        EXPECT(ropes[i](WITH(rope, r, tokens, 0)), FP8BS_OK);
    }
    EXPECT(run_rope8(WITH(rope, r, dim, 64)), FP8BS_ERR_SHAPE);
    EXPECT(run_rope4(WITH(rope, r, page, 24)), FP8BS_ERR_SHAPE);

    /* routing */
    const struct route t = {64, 4, 64, 4, 8, 2, 2, 1, FP8BS_SCORE_SIGMOID, P(void, 0x40000), P(int32_t, 0x60000), 1.0f};
    EXPECT(run_route(WITH(route, t, tokens, -1)), FP8BS_ERR_SHAPE);
    EXPECT(run_route(WITH(route, t, experts, 1025)), FP8BS_ERR_SHAPE);
    EXPECT(run_route(WITH(route, t, stride, 63)), FP8BS_ERR_SHAPE);
    EXPECT(run_route(WITH(route, t, topk, 17)), FP8BS_ERR_SHAPE);
    EXPECT(run_route(WITH(route, t, groups, 7)), FP8BS_ERR_SHAPE);
    EXPECT(run_route(WITH(route, t, open, 9)), FP8BS_ERR_SHAPE);
    EXPECT(run_route(WITH(route, t, top, 3)), FP8BS_ERR_SHAPE);
    EXPECT(run_route(WITH(route, t, scoring, 2)), FP8BS_ERR_SHAPE);
    EXPECT(run_route(WITH(route, t, scale, 0.0f / (t.scale - t.scale))), FP8BS_ERR_SHAPE);
    EXPECT(run_route(WITH(route, t, x, NULL)), FP8BS_ERR_NULL);
    EXPECT(run_route(WITH(route, t, x, P(void, 0x40002))), FP8BS_ERR_ALIGN);
    EXPECT(run_route(WITH(route, t, ids, NULL)), FP8BS_ERR_NULL);
    EXPECT(run_route(WITH(route, t, tokens, 0)), FP8BS_OK);

    /* combination */
    const struct comb c = {8, 4, 2, 64, P(void, 0x40000), P(int32_t, 0x60000), P(void, 0x70000)};
    EXPECT(run_comb(WITH(comb, c, tokens, -1)), FP8BS_ERR_SHAPE);
    EXPECT(run_comb(WITH(comb, c, topk, 1025)), FP8BS_ERR_SHAPE);
    EXPECT(run_comb(WITH(comb, c, n, 0)), FP8BS_ERR_SHAPE);
    EXPECT(run_comb(WITH(comb, c, experts, -1)), FP8BS_ERR_SHAPE);
    EXPECT(run_comb(WITH(comb, c, y, NULL)), FP8BS_ERR_NULL);
    EXPECT(run_comb(WITH(comb, c, out, P(void, 0x70001))), FP8BS_ERR_ALIGN);
    EXPECT(run_comb(WITH(comb, c, ids, P(int32_t, 0x60002))), FP8BS_ERR_ALIGN);
    EXPECT(run_comb(WITH(comb, c, tokens, 0)), FP8BS_OK);

    /* sampling */
    const struct draw d = {1000, 3, 1000, 0, P(void, 0x40000), P(float, 0x50000), P(int32_t, 0x60000)};
    EXPECT(run_draw(WITH(draw, d, rows, -1)), FP8BS_ERR_SHAPE);
    EXPECT(run_draw(WITH(draw, d, vocab, 0)), FP8BS_ERR_SHAPE);
    EXPECT(run_draw(WITH(draw, d, vocab, 1001)), FP8BS_ERR_SHAPE);
    EXPECT(run_draw(WITH(draw, (WITH(draw, d, stride, 2000000)), vocab, 1048577)), FP8BS_ERR_SHAPE);
    EXPECT(run_draw(WITH(draw, d, x, NULL)), FP8BS_ERR_NULL);
    EXPECT(run_draw(WITH(draw, d, u, NULL)), FP8BS_ERR_NULL);
    EXPECT(run_draw(WITH(draw, d, tokens, NULL)), FP8BS_ERR_NULL);
    EXPECT(run_draw(WITH(draw, (WITH(draw, d, f32, 1)), x, P(void, 0x40002))), FP8BS_ERR_ALIGN);
    EXPECT(run_draw(WITH(draw, d, u, P(float, 0x50002))), FP8BS_ERR_ALIGN);
    EXPECT(run_draw(WITH(draw, d, rows, 0)), FP8BS_OK);

    printf("checks %d failures %d\n", checks, failures);
    return failures != 0;
}

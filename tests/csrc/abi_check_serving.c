/*
 * A plain C11 client of the serving-step entry points of include/fp8bs.h
 * (paging plan, 4-bit KV cache, token log probabilities): takes the address of
 * each (a missing export fails the link) and checks their argument validation
 * through the C calling convention.  Every call here is refused, or has
 * nothing to do, before the library touches CUDA, so no GPU is needed.  Prints
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
struct plan { int64_t batch, width, free, page, blocks, tokens; const int32_t *head; int32_t *table, *slots; };

static int run_plan(struct plan p)
{
    const int32_t *in = P(int32_t, 0x10000);
    int32_t *out = P(int32_t, 0x20000);
    return fp8bs_kv_plan(in, in, p.batch, p.table, p.width, in, p.free, p.head, p.page, p.blocks, p.tokens, out, out,
                         p.slots, out, out, out, NULL);
}

struct copy { int64_t tokens, heads, dim, page, blocks, stride; const void *x; const int32_t *slots; };

static int run_append(struct copy c)
{
    return fp4kv_append(c.x, c.stride, c.x, c.stride, c.tokens, c.heads, c.dim, c.slots, P(float, 0x30000),
                        P(float, 0x30000), P(uint8_t, 0x40000), P(uint8_t, 0x50000), c.page, c.blocks, NULL);
}

static int run_gather(struct copy c)
{
    return fp4kv_gather(P(uint8_t, 0x40000), P(uint8_t, 0x50000), c.slots, c.tokens, c.heads, c.dim, c.page, c.blocks,
                        P(float, 0x30000), P(float, 0x30000), (void *)c.x, (void *)c.x, NULL);
}

struct attn {
    int64_t stride, tokens, max_q, width, batch, hq, hkv, dim, page, blocks, max_len, window, ws_bytes;
    const void *q;
    const int32_t *cu;
    float scale;
    void *ws;
};

static int run_attn(struct attn a)
{
    return fp4kv_decode_attention(a.q, a.stride, a.cu, a.tokens, a.max_q, P(uint8_t, 0x40000), P(uint8_t, 0x50000),
                                  P(float, 0x30000), P(float, 0x30000), P(int32_t, 0x60000), a.width,
                                  P(int32_t, 0x70000), a.batch, a.hq, a.hkv, a.dim, a.page, a.blocks, a.max_len,
                                  a.window, a.scale, P(void, 0x80000), NULL, a.ws, a.ws_bytes, NULL);
}

struct lp { const void *x; int f32; int64_t stride, rows, vocab, top; int32_t *ids; float *out; };

static int run_lp(struct lp l)
{
    return fp8bs_token_logprobs(l.x, l.f32, l.stride, l.rows, l.vocab, P(int32_t, 0x10000), l.top, l.out,
                                P(float, 0x20000), l.ids, P(float, 0x30000), NULL);
}

#define WITH(type, base, field, value) ((void)0, (tmp_##type = base, tmp_##type.field = value, tmp_##type))

int main(void)
{
    struct plan tmp_plan;
    struct copy tmp_copy;
    struct attn tmp_attn;
    struct lp tmp_lp;

    /* the paging plan */
    const struct plan p = {4, 16, 64, 16, 64, 8, P(int32_t, 0x30000), P(int32_t, 0x40000), P(int32_t, 0x50000)};
    EXPECT(run_plan(WITH(plan, p, batch, -1)), FP8BS_ERR_SHAPE);
    EXPECT(run_plan(WITH(plan, p, width, 0)), FP8BS_ERR_SHAPE);
    EXPECT(run_plan(WITH(plan, p, free, -1)), FP8BS_ERR_SHAPE);
    EXPECT(run_plan(WITH(plan, p, page, 0)), FP8BS_ERR_SHAPE);
    EXPECT(run_plan(WITH(plan, p, blocks, (int64_t)1 << 28)), FP8BS_ERR_SHAPE);
    EXPECT(run_plan(WITH(plan, p, tokens, -1)), FP8BS_ERR_SHAPE);
    EXPECT(run_plan(WITH(plan, p, head, NULL)), FP8BS_ERR_NULL);
    EXPECT(run_plan(WITH(plan, p, table, NULL)), FP8BS_ERR_NULL);
    EXPECT(run_plan(WITH(plan, p, slots, NULL)), FP8BS_ERR_NULL);
    EXPECT(run_plan(WITH(plan, p, slots, P(int32_t, 0x50002))), FP8BS_ERR_ALIGN);

    /* append and gather */
    const struct copy c = {4, 8, 128, 16, 64, 1024, P(void, 0x10000), P(int32_t, 0x20000)};
    EXPECT(run_append(WITH(copy, c, tokens, -1)), FP8BS_ERR_SHAPE);
    EXPECT(run_append(WITH(copy, c, dim, 96)), FP8BS_ERR_SHAPE);
    EXPECT(run_append(WITH(copy, c, page, 24)), FP8BS_ERR_SHAPE);
    EXPECT(run_append(WITH(copy, c, stride, -8)), FP8BS_ERR_SHAPE);
    EXPECT(run_append(WITH(copy, c, stride, 1028)), FP8BS_ERR_ALIGN);
    EXPECT(run_append(WITH(copy, c, x, NULL)), FP8BS_ERR_NULL);
    EXPECT(run_append(WITH(copy, c, x, P(void, 0x10008))), FP8BS_ERR_ALIGN);
    EXPECT(run_append(WITH(copy, c, tokens, 0)), FP8BS_OK);
    EXPECT(run_gather(WITH(copy, c, heads, 0)), FP8BS_ERR_SHAPE);
    EXPECT(run_gather(WITH(copy, c, blocks, 0)), FP8BS_ERR_SHAPE);
    EXPECT(run_gather(WITH(copy, c, slots, NULL)), FP8BS_ERR_NULL);
    EXPECT(run_gather(WITH(copy, c, slots, P(int32_t, 0x20001))), FP8BS_ERR_ALIGN);
    EXPECT(run_gather(WITH(copy, c, tokens, 0)), FP8BS_OK);

    /* attention and its workspace */
    const int64_t need = fp4kv_attention_ws_bytes(128);
    EXPECT(need > FP4KV_WORKSPACE_COUNTER_BYTES, 1);
    EXPECT(fp4kv_attention_ws_bytes(96), FP8BS_ERR_SHAPE);
    const struct attn a = {4096, 2, 1, 64, 2, 32, 8, 128, 16, 64, 1024, 0, need,
                           P(void, 0x10000), NULL, 0.088f, P(void, 0x90000)};
    EXPECT(run_attn(WITH(attn, a, dim, 32)), FP8BS_ERR_SHAPE);
    EXPECT(run_attn(WITH(attn, a, hq, 36)), FP8BS_ERR_SHAPE);
    EXPECT(run_attn(WITH(attn, a, tokens, 3)), FP8BS_ERR_SHAPE);
    EXPECT(run_attn(WITH(attn, a, max_q, 2)), FP8BS_ERR_SHAPE);
    EXPECT(run_attn(WITH(attn, a, max_len, 1025)), FP8BS_ERR_SHAPE);
    EXPECT(run_attn(WITH(attn, a, window, -1)), FP8BS_ERR_SHAPE);
    EXPECT(run_attn(WITH(attn, a, stride, -8)), FP8BS_ERR_SHAPE);
    EXPECT(run_attn(WITH(attn, a, stride, 4100)), FP8BS_ERR_ALIGN);
    EXPECT(run_attn(WITH(attn, a, scale, 0.0f / (a.scale - a.scale))), FP8BS_ERR_SHAPE);
    EXPECT(run_attn(WITH(attn, a, q, NULL)), FP8BS_ERR_NULL);
    EXPECT(run_attn(WITH(attn, a, ws, NULL)), FP8BS_ERR_NULL);
    EXPECT(run_attn(WITH(attn, a, ws, P(void, 0x90008))), FP8BS_ERR_ALIGN);
    EXPECT(run_attn(WITH(attn, a, ws_bytes, need - 1)), FP8BS_ERR_SHAPE);
    EXPECT(run_attn(WITH(attn, (WITH(attn, a, tokens, 0)), batch, 0)), FP8BS_OK);

    /* log probabilities */
    const struct lp l = {P(void, 0x40000), 0, 1000, 3, 1000, 5, P(int32_t, 0x50000), P(float, 0x60000)};
    EXPECT(run_lp(WITH(lp, l, vocab, 0)), FP8BS_ERR_SHAPE);
    EXPECT(run_lp(WITH(lp, l, stride, 999)), FP8BS_ERR_SHAPE);
    EXPECT(run_lp(WITH(lp, l, top, -1)), FP8BS_ERR_SHAPE);
    EXPECT(run_lp(WITH(lp, l, top, 1001)), FP8BS_ERR_SHAPE);
    EXPECT(run_lp(WITH(lp, l, x, NULL)), FP8BS_ERR_NULL);
    EXPECT(run_lp(WITH(lp, l, ids, NULL)), FP8BS_ERR_NULL);
    EXPECT(run_lp(WITH(lp, l, x, P(void, 0x40001))), FP8BS_ERR_ALIGN);
    EXPECT(run_lp(WITH(lp, (WITH(lp, l, f32, 1)), x, P(void, 0x40002))), FP8BS_ERR_ALIGN);
    EXPECT(run_lp(WITH(lp, l, out, P(float, 0x60001))), FP8BS_ERR_ALIGN);
    EXPECT(run_lp(WITH(lp, l, rows, 0)), FP8BS_OK);

    printf("checks %d failures %d\n", checks, failures);
    return failures != 0;
}

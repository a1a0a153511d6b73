"""One attention layer of a vision-language model held in eight bits, its calls
one behind another as a program makes them: tokens quantized, the QKV product
in 8-bit integers, heads normed and turned by time, height and width, keys and
values appended to an E4M3 cache, attention over it, tokens quantized again and
the attention-out product with the residual.  A prompt of image and text tokens,
then decoding steps behind it, each stage checked against its 64-bit form on
the stage's own inputs, and the steps replayed from a graph."""
import math

import numpy as np
import pytest
import torch

import bf16_gemm_vla_amd as vla
import oracle
import synthetic
from tests.eight_bit_ref import E4M3, append, e8m0_value, quantize_tokens
from tests.gpu_util import bf16_f64, dev, host, zeros_ws
from tests.test_gpu_attention import assert_attention
from tests.test_gpu_axes import check as check_turned
from tests.test_gpu_int8 import check_product

pytestmark = pytest.mark.gpu

HQ, HKV, D, WIDTH = 8, 2, 64, 512
QKV = (HQ + 2 * HKV) * D
PAGE, BLOCK = 32, 16


class Layer:
    def __init__(self, sequences, capacity):
        r = synthetic.rng(59000)
        self.n = sequences
        self.pps = -(-capacity // PAGE)
        self.pages = sequences * self.pps + 2
        self.w = {}
        for name, N, K in (("qkv", QKV, WIDTH), ("out", WIDTH, HQ * D)):
            W = (r.standard_normal((N, K)) * 0.05).astype(np.float32)
            packed, s = torch.empty(N * K, dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda")
            vla.vla_quantize_pack(dev(W), packed, s, N, K, vla.VLA_WFMT_INT8, vla.VLA_LAYOUT_MFMA)
            self.w[name] = (packed, s, *quantize_tokens(W))
        self.bias = synthetic.fp32_to_bf16_bits(r.standard_normal(QKV).astype(np.float32) * 0.1)
        self.qw, self.kw = (synthetic.fp32_to_bf16_bits(1 + 0.2 * r.standard_normal(D).astype(np.float32)) for _ in range(2))
        self.freq = (10000.0 ** (-2.0 * np.arange(D // 2) / D)).astype(np.float32)
        self.axis_of = np.repeat([0, 1, 2], [12, 10, 10]).astype(np.uint8)
        self.table = r.permutation(self.pages)[:sequences * self.pps].reshape(sequences, self.pps).astype(np.int32)
        rows = self.pages * PAGE
        self.cache = [torch.zeros(rows, HKV, D, dtype=torch.uint8, device="cuda") for _ in range(2)]
        self.scales = [torch.zeros(rows // BLOCK, HKV, dtype=torch.uint8, device="cuda") for _ in range(2)]
        self.host_cache = [np.zeros((rows, HKV, D), np.uint8) for _ in range(2)]
        self.host_scales = [np.zeros((rows // BLOCK, HKV), np.uint8) for _ in range(2)]
        self.const = {k: dev(v) for k, v in (("bias", self.bias), ("qw", self.qw), ("kw", self.kw), ("freq", self.freq),
                                             ("axis_of", self.axis_of), ("table", self.table))}

    def buffers(self, T, L):
        e = lambda *s, dtype=torch.int16: torch.empty(*s, dtype=dtype, device="cuda")   # noqa: E731
        n = vla.vla_attn_shared_prefix_e4m3_workspace_bytes(self.n, L, HQ, HKV, D, 0, self.pps * PAGE)
        return {"T": T, "L": L, "x": e(T, WIDTH), "q8": e(T, WIDTH, dtype=torch.int8), "s": e(T, dtype=torch.float32), "qkv": e(T, QKV),
                "pos": e(3, T, dtype=torch.int32), "q": e(T, HQ * D), "k": e(T, HKV * D), "lens": e(self.n, dtype=torch.int32),
                "attn": e(T, HQ * D), "a8": e(T, HQ * D, dtype=torch.int8), "as": e(T, dtype=torch.float32), "y": e(T, WIDTH),
                "ws": zeros_ws(max(vla.vla_gemm_workspace_bytes(T, N, K, vla.VLA_WFMT_INT8) for N, K in ((QKV, WIDTH), (WIDTH, HQ * D)))),
                "aws": torch.empty(n, dtype=torch.uint8, device="cuda"), "aws_n": n}

    def forward(self, b):
        T, L, c, scale = b["T"], b["L"], self.const, 1.0 / math.sqrt(D)
        vla.vla_quantize_tokens_int8(b["x"], b["q8"], b["s"], T, WIDTH)
        vla.vla_gemm_int8(b["q8"], b["s"], *self.w["qkv"][:2], c["bias"], None, b["qkv"], b["ws"], b["ws"].numel(), T, QKV, WIDTH)
        k, v = b["qkv"][:, HQ * D:], b["qkv"][:, (HQ + HKV) * D:]
        vla.vla_qk_norm_rope_axes_append(b["qkv"], k, None, c["qw"], c["kw"], c["freq"], c["axis_of"], b["pos"], None, b["q"], b["k"],
                                         None, None, T, HQ, HKV, D, D, 3, QKV, QKV, 0, HQ * D, HKV * D, 0, vla.VLA_ROPE_HALF, 1.0, 1e-6)
        vla.vla_kv_append_e4m3(b["k"], v, None, c["table"], b["lens"], *self.cache, *self.scales, self.n, L, T, HKV, D, self.pages, PAGE,
                               BLOCK, self.pps, HKV * D, QKV)
        vla.vla_attn_shared_prefix_e4m3(b["q"], *self.cache, *self.scales, None, None, c["table"], b["lens"], b["attn"], b["aws"],
                                        b["aws_n"], self.n, L, HQ, HKV, D, self.pages, PAGE, BLOCK, 0, self.pps, HQ * D, HQ * D, True, scale)
        vla.vla_quantize_tokens_int8(b["attn"], b["a8"], b["as"], T, HQ * D)
        vla.vla_gemm_int8(b["a8"], b["as"], *self.w["out"][:2], None, b["x"], b["y"], b["ws"], b["ws"].numel(), T, WIDTH, HQ * D)

    def check(self, b, lens):
        T, L = b["T"], b["L"]
        get = lambda k: host(b[k], np.uint16 if b[k].dtype == torch.int16 else None)     # noqa: E731
        x, qkv, q, k, attn, y = (get(n) for n in ("x", "qkv", "q", "k", "attn", "y"))
        for codes, s, rows in ((get("q8"), get("s"), x), (get("a8"), get("as"), attn)):
            want_q, want_s = quantize_tokens(bf16_f64(rows))
            assert np.array_equal(codes, want_q) and np.array_equal(s, want_s)
        check_product(qkv, get("q8"), get("s"), *self.w["qkv"][2:], self.bias)
        heads = qkv.reshape(T, HQ + 2 * HKV, D)
        pos = host(b["pos"])
        check_turned(q.reshape(T, HQ, D), heads[:, :HQ], self.qw, self.freq, self.axis_of, pos, D, False, 1.0, 1e-6, "q")
        check_turned(k.reshape(T, HKV, D), heads[:, HQ:HQ + HKV], self.kw, self.freq, self.axis_of, pos, D, False, 1.0, 1e-6, "k")
        for i, rows in enumerate((k.reshape(T, HKV, D), heads[:, HQ + HKV:])):
            append(bf16_f64(rows), np.arange(self.n + 1) * L, self.table, lens, self.host_cache[i], self.host_scales[i], PAGE, BLOCK, L)
            assert np.array_equal(host(self.cache[i]), self.host_cache[i]) and np.array_equal(host(self.scales[i]), self.host_scales[i])
        for seq in range(self.n):
            at = np.arange(lens[seq])
            at = self.table[seq][at // PAGE].astype(np.int64) * PAGE + at % PAGE
            kv = [synthetic.fp32_to_bf16_bits((E4M3[self.host_cache[i][at]] * e8m0_value(self.host_scales[i][at // BLOCK])[..., None]).astype(np.float32))
                  for i in range(2)]
            rows = slice(seq * L, (seq + 1) * L)
            lim = np.clip(np.arange(L) + 1 + lens[seq] - L, 0, lens[seq])
            assert_attention(attn[rows].reshape(L, HQ, D), q[rows].reshape(L, HQ, D), *kv, lim, float(np.float32(1 / math.sqrt(D))), f"sequence {seq}")
        check_product(y, get("a8"), get("as"), *self.w["out"][2:], None, x)


def tokens(seed, T):
    return dev(synthetic.activations(T, WIDTH, 59100 + seed))


def test_layer_prompt_then_decoding_steps_and_their_graph():
    B, L = 3, 70                                   # 7 x 9 patches of a frame and 7 words each
    layer = Layer(B, 100)
    b = layer.buffers(B * L, L)
    patch, word = np.arange(63), np.arange(7) + 9
    pos = np.concatenate([np.stack([0 * patch, patch // 9, patch % 9]), np.stack([word] * 3)], 1)
    b["x"].copy_(tokens(0, B * L))
    b["pos"].copy_(dev(np.tile(pos, (1, B)).astype(np.int32)))
    lens = np.full(B, L)
    b["lens"].copy_(dev(lens.astype(np.int32)))
    layer.forward(b)
    layer.check(b, lens)

    d = layer.buffers(B, 1)
    def step(i):
        d["x"].copy_(tokens(10 + i, B))
        d["pos"].fill_(16 + i)
        d["lens"].fill_(L + 1 + i)
    step(0)
    layer.forward(d)
    layer.check(d, lens + 1)
    start = [t.clone() for t in layer.cache + layer.scales]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward(d)
    for t, s in zip(layer.cache + layer.scales, start):
        t.copy_(s)
    for i in range(1, 5):
        step(i)
        graph.replay()
        layer.check(d, lens + 1 + i)
        again = d["y"].clone()
        d["y"].zero_()
        layer.forward(d)                           # the same rows once more, at once: the same cache and result
        layer.check(d, lens + 1 + i)
        assert torch.equal(d["y"], again)
    vla.vla_workspace_status(d["ws"])


def test_two_layers_side_by_side_on_two_streams():
    """Calls of two layers with buffers of their own, overlapping in time, give what each gives alone."""
    layers = [Layer(2, 64) for _ in range(2)]
    bufs = [layer.buffers(2 * 20, 20) for layer in layers]
    for i, b in enumerate(bufs):
        b["x"].copy_(tokens(30 + i, 40))
        b["pos"].copy_(dev(np.tile(np.arange(20), (3, 2)).astype(np.int32)))
        b["lens"].fill_(20 + 9 * i)
    alone = []
    for layer, b in zip(layers, bufs):
        layer.forward(b)
        torch.cuda.synchronize()
        alone.append([b["y"].clone(), *(t.clone() for t in layer.cache)])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for layer, b, s in zip(layers, bufs, streams):
            with torch.cuda.stream(s):
                b["y"].zero_()
                layer.forward(b)
    torch.cuda.synchronize()
    for layer, b, want in zip(layers, bufs, alone):
        for got, w in zip([b["y"], *layer.cache], want):
            assert torch.equal(got, w)

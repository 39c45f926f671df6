"""The cache operators inside the framework's own paths, against the oracle:
candidate chunks over one prefix (rtv_denoise_shared), the prefix parked in
E4M3 and installed again, and the prefill of more tokens than the tiled
attention takes.

Tolerances are the expert's: fp32 1e-4 max-abs; bf16 relative L2 1e-2 and
max-abs 3e-2 on the chunks.
"""

import numpy as np
import pytest
import torch

from oracle import cache_ops as OC
from oracle import expert as O
from oracle import prefill as OP
from synthetic import (f32_to_bf16_bits, get_config, get_prefill_config, make_noise, make_prefill_weights,
                       make_prefix_embeddings, make_prefix_kv, make_state, make_weights)
from tests.helpers import bf16_tolerance_ok, rel_l2

pytestmark = pytest.mark.gpu


def expert(cfg, max_batch, batch=1):
    from flow_matching_action_dm0_b200 import ActionExpert
    W, kv = make_weights(cfg), make_prefix_kv(cfg, batch=batch)
    ex = ActionExpert(cfg, max_batch=max_batch, max_prefix_len=cfg.prefix_len + 3)   # strides that are not dense
    ex.load(W)
    ex.set_prefix_kv(np.ascontiguousarray(kv))
    return ex, W, kv


def shared_reference(W, cfg, kv, noise, state, n_steps):
    one = kv[:, :, :1]
    return np.concatenate([O.denoise(O.to_f64(W), cfg, noise[i:i + 1], state[None], one, n_steps)
                           for i in range(noise.shape[0])])


@pytest.mark.parametrize("n", [1, 2, 5])
def test_denoise_shared_fp32(cuda_ok, n):
    cfg = get_config("tiny-fp32")
    ex, W, kv = expert(cfg, 5)
    noise, state = make_noise(cfg, batch=5)[:n], make_state(cfg)[0]
    got = ex.denoise_shared(np.ascontiguousarray(noise), state, 4)
    assert np.max(np.abs(got - shared_reference(W, cfg, kv, noise, state, 4))) <= 1e-4
    assert ex.status() == (0, 0)
    ex.close()


@pytest.mark.parametrize("n,variant", [
    (1, {}), (3, {}), (4, {"prefix_len": 37}), (2, {"prefix_len": 1000}), (3, {"n_kv_heads": 2}),
    (3, {"n_kv_heads": 8}), (3, {"head_dim": 128}), (2, {"suffix_mask": "pi0_block"}), (2, {"time_cond": "concat"}),
    (2, {"time_cond": "adarms"}), (5, {"chunk_len": 1}), (3, {"chunk_len": 7, "n_kv_heads": 8})])
def test_denoise_shared_bf16(cuda_ok, n, variant):
    cfg = get_config("pi0-bf16", n_layers=2, **{"prefix_len": 200, **variant})
    ex, W, kv = expert(cfg, max(n, 2), batch=2)       # the chunks share element 0 of the installed two
    assert ex.path == "tcgen05"
    noise, state = np.ascontiguousarray(make_noise(cfg, batch=n)), make_state(cfg)[0]
    got = ex.denoise_shared(noise, state, 2)
    ref = shared_reference(W, cfg, kv, noise, state, 2)
    assert bf16_tolerance_ok(got, ref), (rel_l2(got, ref), np.max(np.abs(got - ref)))
    # the batch's own call still reads both prefixes, and a repeat is bit for bit
    both, states = np.ascontiguousarray(make_noise(cfg, batch=2)), np.ascontiguousarray(make_state(cfg, batch=2))
    own = ex.denoise(both, states, 2)
    ref = O.denoise(O.to_f64(W), cfg, both, states, kv, 2)
    assert bf16_tolerance_ok(own, ref)
    np.testing.assert_array_equal(ex.denoise_shared(noise, state, 2), got)
    assert ex.status() == (0, 0)
    ex.close()


def test_denoise_shared_full_size(cuda_ok):
    """16 candidate chunks of the 18-layer expert over 816 tokens: each agrees with its own denoising."""
    cfg = get_config("pi0-bf16")
    ex, W, kv = expert(cfg, 16)
    noise, state = np.ascontiguousarray(make_noise(cfg, batch=16)), make_state(cfg)[0]
    got = ex.denoise_shared(noise, state, 10)
    for i in (0, 7, 15):
        alone = ex.denoise(np.ascontiguousarray(noise[i:i + 1]), state[None], 10)
        # both within the expert's tolerance of the oracle
        assert bf16_tolerance_ok(got[i:i + 1], alone, rel=2e-2, abs_=6e-2), rel_l2(got[i:i + 1], alone)
    assert ex.status() == (0, 0)
    ex.close()


def test_denoise_shared_refusals(cuda_ok):
    from flow_matching_action_dm0_b200 import ActionExpert, RtvError
    cfg = get_config("tiny-fp32")
    ex, W, kv = expert(cfg, 2)
    noise, state = make_noise(cfg, batch=3), make_state(cfg)[0]
    for n, steps in ((3, 2), (2, 0), (2, 65)):
        with pytest.raises(RtvError) as e:
            ex.denoise_shared(np.ascontiguousarray(noise[:n]), state, steps)
        assert e.value.status == 2
    ex.close()
    ex = ActionExpert(cfg, max_batch=2)
    with pytest.raises(RtvError) as e:
        ex.denoise_shared(np.ascontiguousarray(noise[:2]), state, 2)
    assert e.value.status == 3
    ex.close()


@pytest.mark.parametrize("name,over,batch", [("tiny-fp32", {}, 1), ("pi0-bf16", {"n_layers": 2, "prefix_len": 100}, 2)])
def test_prefix_parked_and_installed_again(cuda_ok, name, over, batch):
    cfg = get_config(name, **over)
    ex, W, kv = expert(cfg, batch, batch=batch)
    codes, scales = ex.get_prefix_kv_quantized(cfg.prefix_len, batch)
    want, size = OC.quantize_rows(np.asarray(kv, np.float64).transpose(0, 1, 2, 4, 3, 5))
    np.testing.assert_array_equal(codes.double().cpu().numpy(), want)
    np.testing.assert_array_equal(scales.double().cpu().numpy(), size)
    noise = np.ascontiguousarray(make_noise(cfg, batch=batch))
    state = np.ascontiguousarray(make_state(cfg, batch=batch))
    ex.set_prefix_kv(np.ascontiguousarray(make_prefix_kv(cfg, batch=batch, seed=9)))   # another observation
    ex.denoise(noise, state, 2)
    ex.set_prefix_kv_quantized(codes, scales)
    got = ex.denoise(noise, state, 2)
    back = np.ascontiguousarray((want * size[..., None]).transpose(0, 1, 2, 4, 3, 5).astype(np.float32))   # exact
    ex.set_prefix_kv(back)
    np.testing.assert_array_equal(got, ex.denoise(noise, state, 2))
    ref = O.denoise(O.to_f64(W), cfg, noise, state, back, 2)
    if cfg.dtype == "f32":
        assert np.max(np.abs(got - ref)) <= 1e-4
    else:
        assert bf16_tolerance_ok(got, ref)
    assert ex.status() == (0, 0)
    ex.close()


def test_parking_refusals(cuda_ok):
    from flow_matching_action_dm0_b200 import ActionExpert, RtvError
    cfg = get_config("tiny-fp32")
    ex, W, kv = expert(cfg, 2)

    def refused(status, call, *a):
        with pytest.raises(RtvError) as e:
            call(*a)
        assert e.value.status == status, str(e.value)

    refused(2, ex.get_prefix_kv_quantized, cfg.prefix_len - 1, 1)
    refused(2, ex.get_prefix_kv_quantized, cfg.prefix_len, 2)
    codes, scales = ex.get_prefix_kv_quantized(cfg.prefix_len, 1)
    refused(1, ex.set_prefix_kv_quantized, codes.cpu(), scales.cpu())
    big = torch.cat([codes.view(torch.uint8)] * 3, dim=2).contiguous()
    refused(2, ex.set_prefix_kv_quantized, big, torch.cat([scales] * 3, dim=2).contiguous())
    with pytest.raises(ValueError):
        ex.set_prefix_kv_quantized(codes[:1].contiguous(), scales[:1].contiguous())
    with pytest.raises(TypeError):
        ex.set_prefix_kv_quantized(codes.float(), scales)
    ex.close()
    ex = ActionExpert(cfg, max_batch=1)
    refused(3, ex.get_prefix_kv_quantized, cfg.prefix_len, 1)
    ex.close()


@pytest.mark.parametrize("n_tokens", [961, 1100])
def test_prefill_past_the_tiled_attention(cuda_ok, n_tokens):
    from flow_matching_action_dm0_b200 import ActionExpert, PrefillStack
    cfg = get_config("pi0-bf16", n_layers=2, prefix_len=n_tokens)
    pc = get_prefill_config("gemma2b-prefill", n_layers=2, width=512, n_q_heads=2, mlp_dim=2048, n_tokens=n_tokens)
    W = make_weights(cfg)
    ex = ActionExpert(cfg, max_batch=1, max_prefix_len=n_tokens + 5)
    ex.load(W)
    pf = PrefillStack(pc, max_tokens=n_tokens)
    stack = {k: f32_to_bf16_bits(v) if v.ndim == 2 else v
             for i in range(2) for k, v in make_prefill_weights(pc, layers=[i]).items()}
    pf.load(stack)
    emb = make_prefix_embeddings(pc, n_tokens=n_tokens)
    noise, state = make_noise(cfg), make_state(cfg)
    got = pf.denoise(ex, emb, noise[0], state[0], 2)
    ref = OP.prefill_denoise(lambda i: make_prefill_weights(pc, layers=[i]), pc, W, cfg, emb, noise, state, 2)[0]
    assert bf16_tolerance_ok(got, ref), (rel_l2(got, ref), np.max(np.abs(got - ref)))
    pf.kv(ex, emb)
    assert rel_l2(ex.denoise(noise, state, 2)[0], got) <= 1e-5
    assert pf.status() == (0, 0) and ex.status() == (0, 0)
    pf.close()
    ex.close()


def test_denoise_shared_shapes(cuda_ok):
    cfg = get_config("tiny-fp32")
    ex, W, kv = expert(cfg, 2)
    noise, state = np.ascontiguousarray(make_noise(cfg, batch=2)), make_state(cfg)[0]
    for bad in ((noise[:, 1:], state), (noise, state[1:]), (noise, np.zeros((2, cfg.state_dim), np.float32))):
        with pytest.raises(ValueError):
            ex.denoise_shared(np.ascontiguousarray(bad[0]), bad[1], 2)
    with pytest.raises(ValueError):
        ex.denoise_shared(noise, state, 2, out=np.zeros_like(noise[:1]))
    ex.close()


def test_park_and_install_on_a_stream_of_their_own(cuda_ok):
    """Nothing is synchronised: memory that another stream's queued work still
    writes is not the parked prefix's, and arrays that are released at once
    are read before their memory serves again."""
    cfg = get_config("pi0-bf16", n_layers=2, prefix_len=100)
    ex, W, kv = expert(cfg, 1)
    noise = torch.from_numpy(np.ascontiguousarray(make_noise(cfg))).cuda()
    state = torch.from_numpy(np.ascontiguousarray(make_state(cfg))).cuda()
    ex.set_prefix_kv_quantized(*ex.get_prefix_kv_quantized(cfg.prefix_len))
    # (a row whose largest value was rounded down to 224 * scale takes half the scale now)
    codes, scales = ex.get_prefix_kv_quantized(cfg.prefix_len)
    want = ex.denoise(noise, state, 2)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        torch.cuda._sleep(20_000_000)                     # the current stream is some 10 ms behind
        junk = torch.empty_like(codes.view(torch.uint8))
        junk.fill_(0x55)
        del junk
        mine = ex.get_prefix_kv_quantized(cfg.prefix_len, stream=stream)
        with torch.cuda.stream(side):
            kept = [t.view(torch.uint8).clone() for t in mine]
        torch.cuda.synchronize()
        same = [bool(torch.equal(x, y.view(torch.uint8))) for x, y in zip(kept, (codes, scales))]
        assert same == [True, True]
        given = codes.clone(), scales.clone()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        ex.set_prefix_kv_quantized(*given, stream=stream)
        del given
        for t in (codes, scales):
            torch.empty_like(t.view(torch.uint8)).fill_(0x11)
        got = ex.denoise(noise, state, 2, stream=stream)
        shared = ex.denoise_shared(noise, state[0], 2, stream=stream)
        torch.cuda.synchronize()
        assert bool(torch.equal(got, want))
        assert bf16_tolerance_ok(shared.cpu().numpy(), want.cpu().numpy(), rel=2e-2, abs_=6e-2)
    assert ex.status() == (0, 0)
    ex.close()


@pytest.mark.parametrize("n_tokens,heads", [(961, 8), (1025, 4)])
def test_prefill_past_the_tiled_attention_with_more_heads_on_one(cuda_ok, n_tokens, heads):
    from flow_matching_action_dm0_b200 import ActionExpert, PrefillStack
    cfg = get_config("pi0-bf16", n_layers=2, prefix_len=n_tokens)
    pc = get_prefill_config("gemma2b-prefill", n_layers=2, width=512, n_q_heads=heads, mlp_dim=1024, n_tokens=n_tokens)
    W = make_weights(cfg)
    ex = ActionExpert(cfg, max_batch=1, max_prefix_len=n_tokens)
    ex.load(W)
    pf = PrefillStack(pc, max_tokens=n_tokens + 70)
    pf.load({k: f32_to_bf16_bits(v) if v.ndim == 2 else v
             for i in range(2) for k, v in make_prefill_weights(pc, layers=[i]).items()})
    emb = make_prefix_embeddings(pc, n_tokens=n_tokens)
    noise, state = make_noise(cfg), make_state(cfg)
    got = pf.denoise(ex, emb, noise[0], state[0], 2)
    ref = OP.prefill_denoise(lambda i: make_prefill_weights(pc, layers=[i]), pc, W, cfg, emb, noise, state, 2)[0]
    assert bf16_tolerance_ok(got, ref), (rel_l2(got, ref), np.max(np.abs(got - ref)))
    assert pf.status() == (0, 0) and ex.status() == (0, 0)
    pf.close()
    ex.close()


def test_a_captured_park_and_install_replay_on_new_values(cuda_ok):
    cfg = get_config("pi0-bf16", n_layers=2, prefix_len=90)
    ex, W, kv = expert(cfg, 1)
    noise, state = np.ascontiguousarray(make_noise(cfg)), np.ascontiguousarray(make_state(cfg))
    first = ex.get_prefix_kv_quantized(cfg.prefix_len)
    ex.set_prefix_kv(np.ascontiguousarray(make_prefix_kv(cfg, seed=9)))
    second = ex.get_prefix_kv_quantized(cfg.prefix_len)
    want = []
    for pair in (first, second):
        ex.set_prefix_kv_quantized(*pair)
        want.append(ex.denoise(noise, state, 2))
    given = [t.clone() for t in first]
    ex.set_prefix_kv_quantized(*given)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ex.set_prefix_kv_quantized(*given)
        parked = ex.get_prefix_kv_quantized(cfg.prefix_len)
    for i in (1, 0, 1):
        for t, new in zip(given, (first, second)[i]):
            t.view(torch.uint8).copy_(new.view(torch.uint8))
        graph.replay()
        np.testing.assert_array_equal(ex.denoise(noise, state, 2), want[i])
        values = [(c.double() * s.double()[..., None]) for c, s in (given, parked)]
        assert bool(torch.equal(*values))          # the same values (a code's scale may be half as large)
    assert ex.status() == (0, 0)
    del graph
    ex.close()

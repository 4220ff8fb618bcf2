"""examples/generate.py: the attention calls and the experts together, step by step against whole
prompts."""
import pytest

torch = pytest.importorskip("torch")

from tests import attn_check as C  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    from quantized_grouped_gemm_router_gb300 import build as B
    B.build()
    from examples import generate
    assert torch.cuda.is_available()
    return generate


def test_steps_match_whole_prompts(ex):
    """After some steps the logits equal those of the texts so far as prompts. Both round to bf16 at the
    same places but in different kernels: a few roundings of 2^-8 in each of two layers."""
    prompts, steps = ex.some_prompts(), 6
    model = ex.small()
    tokens, logits = model.generate(prompts, steps)
    assert tokens.shape == (3, steps)
    assert torch.equal(model.lens.cpu(), torch.tensor([len(p) + steps - 1 for p in prompts], dtype=torch.int32))
    again = model.prefill([p + t[:-1] for p, t in zip(prompts, tokens.tolist())])
    # the residual stream has size ~1 to 3 and ten or so roundings of 2^-9 on average a layer, of random sign
    assert (logits - again).norm() <= 16 * 2.0 ** -9 * again.norm()


def test_same_tokens_twice(ex):
    a, _ = ex.small().generate(ex.some_prompts(1), 4)
    b, _ = ex.small().generate(ex.some_prompts(1), 4)
    assert torch.equal(a, b)


def test_e4m3_cache(ex):
    """The 8-bit cache: the prompts' own logits are the bf16 ones (they do not read the cache), and a
    step's attention is that over the values its codes stand for."""
    import quantized_grouped_gemm_router_gb300 as moe
    prompts = ex.some_prompts(2)
    exact, coded = ex.small(), ex.small(e4m3=True)
    assert torch.equal(exact.prefill(prompts), coded.prefill(prompts))
    block, start = coded.blocks[0], coded.lens.clone()
    q, k, v = block.qkv(coded.embed[torch.tensor([1, 2, 3], device="cuda")])
    moe.kv_append(block.cache, k, v, coded.cu_one, start, coded.table, coded.attn_ws)
    o = moe.attn_decode(block.cache, q, start + 1, coded.table, coded.attn_ws)
    assert moe.read_device_status(coded.attn_ws) == 0
    for b, n in enumerate((start + 1).tolist()):
        for h in range(8):
            kv = [(c[coded.table[b].long(), h // 4].reshape(-1, 64)[:n].view(torch.float8_e4m3fn).float()
                   * s[h // 4]).double().cpu()
                  for c, s in ((block.cache.k, block.cache.k_scale), (block.cache.v, block.cache.v_scale))]
            ref = C.attend(q[b, h:h + 1].cpu().view(torch.bfloat16).double(), *kv, 1 / 8,
                           torch.ones(1, n, dtype=torch.bool))
            C.check(o[b, h:h + 1].contiguous(), None, ref, 11, f"{b} {h}")


def test_refuses_what_does_not_fit(ex):
    model = ex.small()
    with pytest.raises(ValueError):
        model.generate(ex.some_prompts()[:2], 3)
    with pytest.raises(ValueError):
        model.generate([[1] * 255, [1], [2]], 3)


def test_refuses_empty_prompts(ex):
    """A prompt without a token has no last token whose logits could be taken."""
    model = ex.small()
    for prompts in ([[1, 2], [], [3]], [[], [1], [2]], [[1], [2], []]):
        with pytest.raises(ValueError):
            model.generate(prompts, 3)
        with pytest.raises(ValueError):
            model.prefill(prompts)


def test_refuses_no_steps(ex):
    """Fewer than one token cannot be returned; one is the prompts' own."""
    model = ex.small()
    for steps in (0, -3):
        with pytest.raises(ValueError):
            model.generate(ex.some_prompts(), steps)
    assert model.generate(ex.some_prompts(), 1)[0].shape == (3, 1)

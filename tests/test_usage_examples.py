"""The usage shown in README.md and in paged.py runs as it stands, on a step with a prompt, single tokens and a
request that waits, and its served rows are those that training would see."""
import textwrap
from pathlib import Path

import pytest
import torch

import exact_headdim_attention_gb300 as pkg
from exact_headdim_attention_gb300 import paged
from tests import paged_oracle as po
from tests.gpu_util import device_ok
from tests.test_gpu_paged import close

ROOT = Path(__file__).resolve().parent.parent


def readme_step():
    blocks = [b for b in (ROOT / "README.md").read_text().split("```python\n")[1:] if "ffpa_page_plan" in b]
    assert len(blocks) == 1
    code = blocks[0].split("```")[0]
    at = code.index("slots, positions")
    return code[:code.index("q, k = ")], code[at:]        # the frequencies; the step


def docstring_step():
    lines = paged.__doc__.split("\n\n")
    return textwrap.dedent(next(b for b in lines if "ffpa_page_plan" in b))


def test_examples_are_found():
    head, step = readme_step()
    assert "rope_inv_freq" in head
    for code in (head + step, docstring_step()):
        compile(code, "example", "exec")


@pytest.mark.gpu
@pytest.mark.parametrize("source", ["readme", "docstring"])
def test_generation_step_as_shown(source):
    dev = torch.device("cuda:0")
    head, step = readme_step()
    if source == "docstring":
        step = docstring_step()
    g = torch.Generator().manual_seed(31)
    Hq, Hkv, D, page_size, num_tokens, BF = 4, 2, 512, 16, 12, torch.bfloat16
    old, new = [5, 0, 40, 17], [1, 9, 0, 1]
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)   # noqa: E731
    k0, v0, table, _ = po.make_cache(g, old, Hkv, D, page_size, BF, spare=9)
    free = [p for p in range(k0.shape[0]) if p not in set(table.flatten().tolist())]
    k_cache, v_cache = k0.to(dev), v0.to(dev)
    qkv = torch.randn(num_tokens, Hq + 2 * Hkv, D, generator=g).to(BF).to(dev)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    q_weight, k_weight = (1 + 0.2 * torch.randn(2, D, generator=g)).to(BF).to(dev)
    names = {n: getattr(pkg, n) for n in pkg.__dict__ if n.startswith(("ffpa_", "rope_"))}
    scope = dict(names, ffpa=pkg, table=table.to(dev), lens=i32(*old), new_lens=i32(*new), new=i32(*new), free_pages=i32(*free),
                 free=i32(*free), free_count=i32(len(free)), page_size=page_size, page=page_size, num_tokens=num_tokens,
                 tokens=num_tokens, q=q, k=k, v=v, k_cache=k_cache, v_cache=v_cache, q_weight=q_weight, k_weight=k_weight)
    exec(head, scope)
    exec(step, scope)
    device_ok()
    # what training gives for these rows: the same norm, angles and scale
    qt, kt = pkg.ffpa_qk_norm_rope(q, k, scope["positions"], scope["inv_freq"], q_weight, k_weight, rope_scale=scope["scale"])
    assert scope["scale"] > 1.2 and torch.equal(scope["q"], qt)
    rows = scope["slots"][:sum(new)]
    assert torch.equal(k_cache.view(-1, Hkv, D)[rows], kt[:sum(new)])
    last = [0, 9, 9, 10]                                   # request 2 waits
    ref = po.decode(qt[last].cpu(), k_cache.cpu(), v_cache.cpu(), scope["table"].cpu(), scope["lens"].cpu())
    o = scope["o"]
    assert scope["lens"].tolist() == [6, 9, 40, 18]
    # (rope_scale makes the rotated rows 1.2 times as long: scores stay below 8)
    for b in (0, 1, 3):
        close(o[b], ref[0][b], ref[2][b], f"request {b}")

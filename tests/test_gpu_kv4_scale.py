"""The two rules of a 4-bit group's scale: a / 7 as an f32 quotient, or a times the f32 next to 1 / 7."""
import numpy as np
import pytest

from tests._kvrows import bf16_round, kv4_values


def _apart():
    """Rows of 64 whose two groups' scales differ between the rules: a next to 7 times a border of bf16."""
    rng = np.random.default_rng(11)
    h = (1 + (2 * rng.integers(0, 128, 20000) + 1) / 256).astype(np.float64)      # 9 bits: between two bf16
    a = (7 * h * 2.0 ** rng.integers(-100, 100, 20000)).astype(np.float32)
    a = np.concatenate([a, np.nextafter(a, np.float32(0)), np.nextafter(a, np.float32(np.inf))])
    a = a[bf16_round(a / np.float32(7)) != bf16_round(a * (np.float32(1) / np.float32(7)))]
    a = a[:len(a) // 2 * 2].reshape(-1, 2, 1)
    x = rng.uniform(-0.99, 0.99, (len(a), 2, 32)).astype(np.float32) * a
    x[:, :, 7] = a[:, :, 0]
    return x.reshape(-1, 64)


def _product_values(x):
    """What the product rule stores, of f32 rows [n, 64]."""
    g = x.reshape(-1, 32)
    s = bf16_round(np.abs(g).max(axis=1) * (np.float32(1) / np.float32(7)))
    s = np.where(s < np.float32(2.0 ** -126), np.float32(0), s).astype(np.float64)[:, None]
    return (np.rint(np.divide(g.astype(np.float64), s, out=np.zeros(g.shape), where=s > 0)) * s).reshape(x.shape)


def _stored(rows, **kw):
    import torch
    import transformer_decoder_kv_b200 as pkg
    n = len(rows)
    view = pkg.KvView(1, 64, -(-n // 64), 1)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    batch = pkg.KvRows(1, i32(n), None, i32(0, n), n, n)
    cache = torch.empty(pkg.kv4_bytes(view), dtype=torch.uint8, device="cuda")
    x = torch.from_numpy(rows).cuda()
    pkg.kv4_write(view, batch, x, -x, cache, **kw)
    k, v = torch.empty_like(x), torch.empty_like(x)
    pkg.kv4_read(view, batch, cache, k, v)
    torch.cuda.synchronize()
    assert torch.equal(k, -v)
    return k.cpu().numpy()


def test_the_rules_differ_at_borders_of_bf16_only():
    x = _apart()
    assert len(x) > 500
    ratio = np.abs(kv4_values(x)).max() / np.abs(_product_values(x)).max()
    assert 1 - 2.0 ** -7 <= ratio <= 1 + 2.0 ** -7
    y = np.random.default_rng(0).standard_normal((4096, 64)).astype(np.float32)
    assert (kv4_values(y) != _product_values(y)).any(axis=1).sum() <= 4       # 1 in 60,000 groups


@pytest.mark.gpu
def test_each_rule_stores_its_own_codes():
    x = np.concatenate([_apart(), np.random.default_rng(1).standard_normal((40000, 64)).astype(np.float32),
                        np.full((1, 64), 3.4e38, np.float32), np.full((1, 64), 1e-40, np.float32),
                        np.full((1, 64), 8e-38, np.float32)])
    assert np.array_equal(_stored(x), kv4_values(x))
    assert np.array_equal(_stored(x, scale="quotient"), kv4_values(x))
    assert np.array_equal(_stored(x, scale="product"), _product_values(x))


@pytest.mark.gpu
def test_the_product_rule_is_what_torch_stores():
    """The same rows quantised with elementary torch operations on the GPU, max / 7.0 among them."""
    import torch
    x = np.concatenate([_apart(), np.random.default_rng(2).standard_normal((40000, 64)).astype(np.float32)])
    g = torch.from_numpy(x).cuda().view(-1, 32)
    s = (g.abs().amax(-1, keepdim=True) / 7.0).to(torch.bfloat16)
    s = torch.where(s < 2.0 ** -126, torch.zeros_like(s), s).double()
    want = torch.round(g.double() / s) * s
    assert np.array_equal(_stored(x, scale="product"), want.view(x.shape).float().cpu().numpy())

"""What the compiled binding refuses before anything is enqueued: tensors that the library behind it
would see as bare pointers."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

T, HQ, HK, D, B, PAGE, PAGES = 4, 4, 2, 64, 2, 16, 6


@pytest.fixture(scope="module")
def lb():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bit_weight_gemv_gb300 as lb
    lb.lowbit_device_error()
    yield lb
    torch.cuda.synchronize()
    assert lb.lowbit_device_error() == 0


def bf16(*shape):
    return torch.ones(shape, dtype=torch.bfloat16, device="cuda")


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def append_args(lb):
    return dict(q=bf16(T, HQ, D), k=bf16(T, HK, D), v=bf16(T, HK, D), rope=torch.ones((40, D), device="cuda"),
                cu_q=i32([0, 1, T]), kv_lens=i32([5, 20]), block_table=i32([[0, 1], [2, 3]]),
                cache=lb.lowbit_paged_cache(bf16(PAGES, PAGE, HK, D), bf16(PAGES, PAGE, HK, D)), q_out=bf16(T, HQ, D))


def attention_args(lb):
    a = append_args(lb)
    need = lb.lowbit_paged_attention_workspace_bytes(T, B, HQ, HK, D)
    return dict(q=a["q"], cache=a["cache"], cu_q=a["cu_q"], kv_lens=a["kv_lens"], block_table=a["block_table"],
                out=bf16(T, HQ, D), workspace=torch.zeros(need, dtype=torch.uint8, device="cuda"),
                lse=torch.zeros((T, HQ), device="cuda"))


def sample_args(lb):
    f = dict(device="cuda")
    return dict(logits=torch.zeros((3, 50), **f), u=torch.zeros(3, **f), ids=i32([0, 0, 0]), temperature=torch.ones(3, **f),
                top_k=i32([0, 0, 0]), top_p=torch.ones(3, **f), min_p=torch.zeros(3, **f), id_map=i32([0] * 50),
                logprob=torch.zeros(3, **f), kept=i32([0, 0, 0]))


BATCH = [("cu_q", lambda t: t.long(), TypeError), ("cu_q", lambda t: t[:-1].contiguous(), ValueError),
         ("cu_q", lambda t: t.cpu(), TypeError), ("kv_lens", lambda t: t.float(), TypeError),
         ("kv_lens", lambda t: torch.stack([t, t], 1)[:, 0], TypeError), ("kv_lens", lambda t: t[:1].contiguous(), ValueError),
         ("block_table", lambda t: t[:1], ValueError), ("block_table", lambda t: t.t(), ValueError),
         ("block_table", lambda t: t.reshape(-1), ValueError), ("block_table", lambda t: t.long(), TypeError),
         ("block_table", lambda t: None, TypeError)]


@pytest.mark.parametrize("name,change,kind", BATCH + [
    ("q", lambda t: t.float(), TypeError), ("q", lambda t: t.cpu(), TypeError), ("q", lambda t: None, ValueError),
    ("q_out", lambda t: None, ValueError), ("q_out", lambda t: t[:-1], ValueError), ("q_out", lambda t: t.half(), TypeError),
    ("q_out", lambda t: t.transpose(0, 1), TypeError), ("q", lambda t: t[:-1], ValueError),
    ("q", lambda t: t[..., ::2], ValueError), ("q", lambda t: t.transpose(0, 1).contiguous().transpose(0, 1), ValueError),
    ("k", lambda t: t[:, :1], ValueError), ("k", lambda t: t[..., :32], ValueError), ("v", lambda t: t[:-1], ValueError),
    ("v", lambda t: t.view(T, -1), ValueError), ("k", lambda t: [1], TypeError), ("rope", lambda t: t.double(), TypeError),
    ("rope", lambda t: t.view(-1), ValueError), ("rope", lambda t: t.t(), TypeError)])
def test_append(lb, name, change, kind):
    a = append_args(lb)
    a[name] = change(a[name])
    with pytest.raises(kind):
        lb.lowbit_kv_append(**a)


@pytest.mark.parametrize("name,change,kind", BATCH + [
    ("q", lambda t: None, TypeError), ("q", lambda t: t.float(), TypeError), ("q", lambda t: t[..., :32], ValueError),
    ("q", lambda t: t.transpose(0, 1).contiguous().transpose(0, 1), ValueError), ("out", lambda t: t[:-1], ValueError),
    ("out", lambda t: t.float(), TypeError), ("out", lambda t: None, TypeError),
    ("out", lambda t: torch.cat([t, t], 2)[..., :D], TypeError), ("workspace", lambda t: t.view(torch.int16), TypeError),
    ("workspace", lambda t: t.cpu(), TypeError), ("lse", lambda t: t.half(), TypeError), ("lse", lambda t: t[:-1], ValueError),
    ("lse", lambda t: t.t(), TypeError)])
def test_attention(lb, name, change, kind):
    a = attention_args(lb)
    a[name] = change(a[name])
    with pytest.raises(kind):
        lb.lowbit_paged_attention(**a)


@pytest.mark.parametrize("kw,kind", [(dict(window=2 ** 40), ValueError), (dict(window=1.5), TypeError),
                                     (dict(window="x"), TypeError), (dict(scale="x"), TypeError), (dict(stream="x"), Exception)])
def test_attention_settings(lb, kw, kind):
    with pytest.raises(kind):
        lb.lowbit_paged_attention(**attention_args(lb), **kw)


def test_library_statuses_come_back_as_errors(lb):
    a = attention_args(lb)
    for kw, status in ((dict(window=-1), 2), (dict(workspace=a["workspace"][:64]), 4), (dict(scale=float("nan")), 1),
                       (dict(workspace=a["workspace"][8:]), 4)):
        with pytest.raises(lb.LowbitError) as e:
            lb.lowbit_paged_attention(**(a | kw))
        assert e.value.status == status
    a = append_args(lb)
    product = bf16(T, HQ + 2 * HK, D)
    for kw, status in ((dict(rope=torch.ones((40, 24), device="cuda")), 2), (dict(rope=torch.ones((0, D), device="cuda")), 1),
                       (dict(q=product[:, :HQ], q_out=torch.as_strided(product, (T, HQ, D), (HQ * D, D, 1))), 1)):
        with pytest.raises(lb.LowbitError) as e:
            lb.lowbit_kv_append(**(a | kw))
        assert e.value.status == status


@pytest.mark.parametrize("name,change,kind", [
    ("logits", lambda t: t.half(), TypeError), ("logits", lambda t: t.cpu(), TypeError), ("logits", lambda t: t[0], TypeError),
    ("logits", lambda t: t.t().contiguous().t(), ValueError), ("logits", lambda t: None, TypeError),
    ("u", lambda t: t.double(), TypeError), ("u", lambda t: t[:-1], ValueError), ("u", lambda t: None, TypeError),
    ("ids", lambda t: t.long(), TypeError), ("ids", lambda t: t[:-1], ValueError), ("temperature", lambda t: t[:1], ValueError),
    ("top_k", lambda t: t.float(), TypeError), ("top_p", lambda t: 0.9, TypeError), ("min_p", lambda t: t.cpu(), TypeError),
    ("id_map", lambda t: t[:-1], ValueError), ("logprob", lambda t: t.bfloat16(), TypeError), ("kept", lambda t: t[::2], Exception)])
def test_sample(lb, name, change, kind):
    a = sample_args(lb)
    a[name] = change(a[name])
    with pytest.raises(kind):
        lb.lowbit_sample(**a)


def test_caches(lb):
    good = bf16(PAGES, PAGE, HK, D)
    fp8 = good.to(torch.float8_e4m3fn)
    one = torch.ones(HK, device="cuda")
    for k, v, ks, vs, kind in ((good.cpu(), good.cpu(), None, None, TypeError), (good.float(), good.float(), None, None, TypeError),
                               (good[0], good[0], None, None, TypeError), (good[..., ::2], good[..., ::2], None, None, TypeError),
                               (good, good[:-1], None, None, ValueError), (good, fp8, None, None, ValueError),
                               (good, good.transpose(1, 2).contiguous().transpose(1, 2), None, None, ValueError),
                               (good, good, one, None, ValueError), (fp8, fp8, one[:1], None, ValueError),
                               (fp8, fp8, None, one.half(), TypeError)):
        with pytest.raises(kind):
            lb.lowbit_paged_cache(k, v, ks, vs)

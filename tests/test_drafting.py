"""examples/transformer_layer.py: the operators for drafted tokens together, as
they are used: trees of drafts, their verification, the caches."""
import pytest

from test_transformer_layer import example  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def models(example):  # noqa: F811
    import torch
    torch.manual_seed(0)
    model, drafter = example.Decoder().cuda().bfloat16(), example.Decoder(layers=1, width=128, heads=2, heads_kv=1).cuda().bfloat16()
    example.train(model, 60), example.train(drafter, 60)
    return model.eval(), drafter.eval()


def bound(most):
    """What two ways of computing a logit may differ by: each of two layers' five results is rounded to 2^-8 of itself."""
    return 2 * 2 * 5 * 2.0 ** -8 * max(most, 1.0)


def test_a_tree_from_the_cache_agrees_with_whole_sequences(example, models):  # noqa: F811
    import torch
    model = models[0]
    g = torch.Generator(device="cuda").manual_seed(2)
    s = example.sequences(3, 30, 64, g)
    caches = model.caches(3, 60, model.head.weight)
    lengths = torch.zeros(3, dtype=torch.int32, device="cuda")
    whole = model(s).detach().float()
    chain = model.tree(s[:, :20], caches, lengths).float()
    assert float((chain - whole[:, :20]).abs().max()) < bound(float(whole.abs().max()))
    # two branches after token 20: the sequence's own, and other tokens
    parents = torch.tensor([[-1, 0, 0, 1, 2, 3]] * 3, dtype=torch.int32, device="cuda")
    other = torch.randint(64, (3, 2), generator=g, device="cuda")
    tokens = torch.stack([s[:, 20], s[:, 21], other[:, 0], s[:, 22], other[:, 1], s[:, 23]], 1)
    tree = model.tree(tokens, caches, lengths + 20, parents).float()
    beside = model(torch.cat([s[:, :21], other], 1)).detach().float()
    for node, at, rows in ((0, 20, whole), (1, 21, whole), (3, 22, whole), (5, 23, whole), (2, 21, beside), (4, 22, beside)):
        assert float((tree[:, node] - rows[:, at]).abs().max()) < bound(float(whole.abs().max())), node


def test_greedy_drafting_gives_what_the_model_alone_would(example, models):  # noqa: F811
    """Each token is the largest of the whole sequence's logits, or as near to it as the two ways of computing them are;
    and a draft stands whenever it is that token."""
    import torch
    model, drafter = models
    prompts = example.sequences(4, 12, 64, torch.Generator(device="cuda").manual_seed(5))
    new, stood = example.speculate(model, drafter, prompts, 6, greedy=True)
    assert stood > 0 and sum(map(len, new)) == stood + 4 * 6
    for prompt, tokens in zip(prompts.tolist(), new):
        logits = model(torch.tensor([prompt + tokens], device="cuda")).detach().float()[0, len(prompt) - 1:-1]
        chosen = logits.gather(1, torch.tensor(tokens, device="cuda")[:, None])[:, 0]
        assert bool((chosen >= logits.amax(1) - 2 * bound(float(logits.abs().max()))).all())


def test_a_drafter_that_is_the_model_stands_throughout(example, models):  # noqa: F811
    """Drafts drawn from the target's own distribution stand but for the two ways of computing it (trees of different
    sizes): logits within 0.34 make each stand with a probability of a half at least."""
    import torch
    model = models[0]
    prompts = example.sequences(4, 12, 64, torch.Generator(device="cuda").manual_seed(6))
    new, stood = example.speculate(model, model, prompts, 5, width=1, depth=4)
    assert stood >= 0.5 * 4 * 5 * 4 and all(0 <= t < 64 for tokens in new for t in tokens)


def test_the_same_seed_gives_the_same_tokens(example, models):  # noqa: F811
    import torch
    prompts = example.sequences(4, 12, 64, torch.Generator(device="cuda").manual_seed(7))
    first, again, other = (example.speculate(*models, prompts, 5, seed=seed) for seed in (3, 3, 4))
    assert first == again and first != other


@pytest.mark.parametrize("length", (1, 2, 128, 129, 130, 300))
def test_prompts_of_any_length(example, models, length):  # noqa: F811
    """One token, as many as a tree has nodes, and more: the tokens are the largest logits of the whole sequence's."""
    import torch
    model, drafter = models
    prompts = example.sequences(2, length, 64, torch.Generator(device="cuda").manual_seed(length))
    new, _ = example.speculate(model, drafter, prompts, 3, greedy=True)
    for prompt, tokens in zip(prompts.tolist(), new):
        assert len(tokens) >= 3
        logits = model(torch.tensor([prompt + tokens], device="cuda")).detach().float()[0, len(prompt) - 1:-1]
        chosen = logits.gather(1, torch.tensor(tokens, device="cuda")[:, None])[:, 0]
        assert bool((chosen >= logits.amax(1) - 2 * bound(float(logits.abs().max()))).all())
